// Writing, reading back and committing rows of the paged key/value cache:
// kv_append, qkv_norm_rope_append, kv_gather, kv_commit (include/qlin.h).
//
// All four move data; a pass reads and writes each byte once and the memory
// system is the bound.  A wave handles one head of four consecutive tokens,
// 16 lanes to a row of D elements (D / 16 each).  Four tokens are what the
// cache's V order keeps side by side: when their slots are one aligned
// quad of a page -- every quad of a prompt that starts on one -- the wave
// transposes its 4 x 4 units between the four rows and stores whole dwords;
// otherwise each lane stores its elements one by one.  Reading codes needs no
// transpose: a lane reads all four tokens' elements, which the other rows of
// its wave mostly need too, in wide loads and keeps its own.
#include "kv_cache.hpp"

namespace qlin {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;   // waves per block

// --------------------------------------------------------------------------
// 16-lane row reductions (DPP: xor 1, xor 2, mirrors of 8 and 16)
// --------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF,
                                                            0xF, true));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  return v;
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_mov_dpp(int(u), CTRL, 0xF, 0xF, true));
  const uint32_t hi = uint32_t(__builtin_amdgcn_mov_dpp(int(u >> 32), CTRL, 0xF, 0xF, true));
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ double row_sum(double v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  return v;
}
__device__ __forceinline__ float fma_of(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fma_of(double a, double b, double c) { return __builtin_fma(a, b, c); }
__device__ __forceinline__ float rsqrt_of(float v) { return __builtin_amdgcn_rsqf(v); }
__device__ __forceinline__ double rsqrt_of(double v) {
  // One step of Newton's method from the instruction's 23 bits; v may
  // lie outside of binary32's range (rows of below 1e-19 with eps = 0, or above
  // 1e19).  0 and infinity: infinity and 0.
  const double r = __builtin_amdgcn_rsq(v);
  const double y = r * (1.5 - 0.5 * v * r * r);
  return r > 0.0 && r < __builtin_inf() ? y : r;
}
__device__ __forceinline__ float row_max(float v) {
  v = __builtin_fmaxf(v, dpp<0xB1>(v));
  v = __builtin_fmaxf(v, dpp<0x4E>(v));
  v = __builtin_fmaxf(v, dpp<0x141>(v));
  v = __builtin_fmaxf(v, dpp<0x140>(v));
  return v;
}

// --------------------------------------------------------------------------
// 4 x 4 transposes between the four rows of a wave (lanes 16 apart).  Both
// are their own inverse.
// --------------------------------------------------------------------------
// Byte k of the result is byte j of row k's word; j is this lane's row.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t w, int j) {
  const uint32_t a = __shfl_xor(w, 16, 64), b = __shfl_xor(w, 32, 64), c = __shfl_xor(w, 48, 64);
  const uint32_t sel = 0x0C0C0000u | (j & 1 ? uint32_t(j | (4 + j) << 8) : uint32_t(4 + j | j << 8));
  const uint32_t near = __builtin_amdgcn_perm(w, a, sel);   // rows j & ~1, j | 1
  const uint32_t far = __builtin_amdgcn_perm(b, c, sel);
  return j & 2 ? far | near << 16 : near | far << 16;
}
// Half k of the result (two words) is half j of row k's two words.
__device__ __forceinline__ uint2 transpose_halves(uint32_t w0, uint32_t w1, int j) {
  const uint32_t mine = j & 2 ? w1 : w0, other = j & 2 ? w0 : w1;
  const uint32_t a = __shfl_xor(mine, 16, 64), b = __shfl_xor(other, 32, 64),
                 c = __shfl_xor(other, 48, 64);
  const uint32_t sel = j & 1 ? 0x07060302u : 0x01000504u;
  const uint32_t near = __builtin_amdgcn_perm(mine, a, sel), far = __builtin_amdgcn_perm(b, c, sel);
  return j & 2 ? make_uint2(far, near) : make_uint2(near, far);
}

// --------------------------------------------------------------------------
// Rows in registers
// --------------------------------------------------------------------------
// Two or four floats from an address that is a multiple of 4 bytes.
__device__ __forceinline__ f32x2 load2(const float* p) {
  typedef f32x2 unaligned __attribute__((aligned(4)));
  return *reinterpret_cast<const unaligned*>(p);
}
__device__ __forceinline__ f32x4 load4(const float* p) {
  typedef f32x4 unaligned __attribute__((aligned(4)));
  return *reinterpret_cast<const unaligned*>(p);
}

template <bool F32, int N>
__device__ __forceinline__ void load_row(const void* base, int64_t off, float (&x)[N]) {
  if constexpr (F32) {
    const float* p = static_cast<const float*>(base) + off;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + off;
    uint32_t w[N / 2];
    if constexpr (N == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    *static_cast<uint32_t*>(p) = w[0];
  } else if constexpr (N == 2) {
    *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      static_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

template <int N>
__device__ __forceinline__ void store_row_bf16(void* base, int64_t off, const float (&x)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  store_words(static_cast<uint16_t*>(base) + off, w);
}

// What a lane holds of an encoded row: `w` the row's bytes in order (16-bit
// elements, 8-bit codes, or pairs of 4-bit codes), the E4M3 scale of the
// group its elements lie in, and the row's stored exponent.
template <int FMT, int D>
struct EncRow {
  static constexpr int N = D / 16;                                      // elements per lane
  static constexpr int kBytes = KvLayout<FMT, D>::kRow / 16;            // of the row per lane
  static constexpr int kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];
  uint32_t scale, exp;
};

// Row exponent for a row of maximum amax (a bit pattern of a non-negative
// float): the smallest e with amax <= Q 2^e, Q = 448 = 1.75 * 2^8 or
// 2688 = 1.3125 * 2^11, as e + 127; at least kKvExpMin, which rows of zeros take
// (with an e of 0 their weight in an attention would be that of rows that large,
// and small rows beside them would lose their bits).
template <int FMT>
__device__ __forceinline__ uint32_t row_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax), m = u & 0x7FFFFFu;
  constexpr int shift = FMT == QL_KV_E4M3 ? 8 : 11;
  constexpr uint32_t top = FMT == QL_KV_E4M3 ? 0x600000u : 0x280000u;
  const int b = int(u >> 23) - shift + (m > top ? 1 : 0);
  return uint32_t(b < kKvExpMin ? kKvExpMin : b);
}

// A value in binary32 that rounds on to fewer bits as v itself does: where it
// is not exact the last bit is set (and what was rounded up is taken back).
__device__ __forceinline__ float sticky(float v) { return v; }
__device__ __forceinline__ float sticky(double v) {
  const float f = static_cast<float>(v);
  const double back = f;
  uint32_t u = __float_as_uint(f);
  if (__builtin_fabs(back) > __builtin_fabs(v)) u -= 1;
  return __uint_as_float(back != v ? u | 1u : u);
}
template <typename T>
__device__ __forceinline__ T greater(T a, T b) {
  if constexpr (sizeof(T) == 8) return __builtin_fmax(a, b);
  else return __builtin_fmaxf(a, b);
}

// Encodes this lane's N elements (binary32, or keys in binary64) of a row held
// by 16 lanes.  An infinity takes the largest code; a NaN stays one (8-bit: its
// own code; 4-bit: its group's scale).
template <int FMT, int D, typename T>
__device__ __forceinline__ EncRow<FMT, D> encode_row(const T (&v)[D / 16]) {
  constexpr int N = D / 16;
  float x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = sticky(v[i]);
  EncRow<FMT, D> r;
  r.scale = 0;
  if constexpr (FMT == QL_KV_BF16) {
    r.exp = 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) r.w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    return r;
  } else {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) a = __builtin_fmaxf(a, __builtin_fabsf(x[i]));
    const float amax = row_max(a);
    r.exp = row_exponent<FMT>(amax);
    const float p = __uint_as_float((254u - r.exp) << 23);   // 2^-e
    float y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = x[i] * p;
    if constexpr (FMT == QL_KV_E4M3) {
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = y[i] > 448.0f ? 448.0f : y[i] < -448.0f ? -448.0f : y[i];
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
        r.w[i] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], v, true));
      }
    } else {
      // group maximum over 16 elements: 16 / N lanes
      T g = 0;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < N; ++i) g = greater<T>(g, std::fabs(v[i])), nan |= x[i] != x[i];
      float bad = nan ? 1.0f : 0.0f;
      if constexpr (N < 16) {
        g = greater<T>(g, dpp<0xB1>(g));
        bad = __builtin_fmaxf(bad, dpp<0xB1>(bad));
      }
      if constexpr (N < 8) {
        g = greater<T>(g, dpp<0x4E>(g));
        bad = __builtin_fmaxf(bad, dpp<0x4E>(bad));
      }
      const float q = __builtin_fminf(static_cast<float>(g * T(p) / T(6)), 448.0f);
      const uint32_t sc = __builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0xFFu;
      const float sv = __builtin_amdgcn_cvt_f32_fp8(int(sc), 0);
      const float inv = sv > 0.0f ? 1.0f / sv : 0.0f;
      r.scale = bad > 0.0f ? 0x7Fu : sc;
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = static_cast<float>(v[i] * T(p) * T(inv));
#pragma unroll
      for (int i = 0; i < EncRow<FMT, D>::kWords; ++i) {
        uint32_t v = 0;
        v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, y[8 * i], y[8 * i + 1], 1.0f, 0);
        v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, y[8 * i + 2], y[8 * i + 3], 1.0f, 1);
        if constexpr (N > 4) {
          v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, y[8 * i + 4], y[8 * i + 5], 1.0f, 2);
          v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, y[8 * i + 6], y[8 * i + 7], 1.0f, 3);
        }
        r.w[i] = v;
      }
    }
    return r;
  }
}

// Where a token's row lies: the block's codes and scales, and the token in it.
struct Place {
  uint8_t* codes;
  uint8_t* scales;
  int t;
};
template <int FMT, int D>
__device__ __forceinline__ Place place_of(const KvGeom& g, int64_t slot, int head) {
  using L = KvLayout<FMT, D>;
  const int64_t page = slot >> g.page_shift;
  const int in = int(slot & ((int64_t(1) << g.page_shift) - 1));
  const int64_t block = kv_block(g, page, head, in >> 4);
  return {g.codes + block * L::kCodes, g.scales + block * L::kScales, in & 15};
}
__device__ __forceinline__ bool slot_ok(const KvGeom& g, int64_t slot) {
  return slot >= 0 && (slot >> g.page_shift) < g.n_pages;
}

// The first of a block's four tokens: quads of tokens start where those of the
// first token's page do, so that the tokens of one prompt fall into whole
// quads wherever it starts (0 to 3 tokens before the first one are missing).
__device__ __forceinline__ int64_t first_token(const int64_t* slots) {
  return int64_t(blockIdx.x) * 4 - (slots[0] & 3);
}
// Blocks of four tokens that cover `tokens` tokens wherever the first lies.
unsigned quads(int64_t tokens) { return unsigned((tokens + 6) / 4); }

// Whether the wave's four tokens are one aligned quad of the cache; the same
// in every lane (all lanes must call).
__device__ __forceinline__ bool whole_quad(int64_t slot, bool ok, int j) {
  const int64_t first = __shfl(slot, 0, 64);
  return __all(ok && slot == first + j && (first & 3) == 0);
}

template <int FMT, int D>
__device__ __forceinline__ void store_k(const Place& p, int i, const EncRow<FMT, D>& r) {
  using L = KvLayout<FMT, D>;
  using E = EncRow<FMT, D>;
  if constexpr (E::kBytes == 2) {
    *reinterpret_cast<uint16_t*>(p.codes + L::k_code(p.t, 2 * i)) = uint16_t(r.w[0]);
  } else if constexpr (E::kBytes <= 16) {
    store_words(p.codes + L::k_code(p.t, E::kBytes * i), r.w);
  } else {
#pragma unroll
    for (int c = 0; c < E::kBytes / 16; ++c)
      *reinterpret_cast<uint4*>(p.codes + L::k_code(p.t, E::kBytes * i + 16 * c)) =
          make_uint4(r.w[4 * c], r.w[4 * c + 1], r.w[4 * c + 2], r.w[4 * c + 3]);
  }
  if constexpr (FMT == QL_KV_NVFP4) {
    constexpr int lanes = 16 / E::N;   // lanes of a group
    if (i % lanes == 0) p.scales[L::k_scale(p.t, i / lanes)] = uint8_t(r.scale);
  }
  if constexpr (FMT != QL_KV_BF16) {
    if (i == 0) p.scales[L::k_exp(p.t)] = uint8_t(r.exp);
  }
}

// `quad`: the wave's rows are one aligned quad (all lanes active then);
// `ok`: this lane's row is stored.
template <int FMT, int D>
__device__ __forceinline__ void store_v(const Place& p, int i, int j, bool quad, bool ok,
                                        const EncRow<FMT, D>& r) {
  using L = KvLayout<FMT, D>;
  using E = EncRow<FMT, D>;
  if (quad) {
    const int t0 = p.t & ~3;
    if constexpr (FMT == QL_KV_BF16) {
#pragma unroll
      for (int w = 0; w < E::kWords / 2; ++w) {
        const uint2 v = transpose_halves(r.w[2 * w], r.w[2 * w + 1], j);
        *reinterpret_cast<uint2*>(p.codes + L::v_code(t0, E::N * i + 4 * w + j)) = v;
      }
    } else {
#pragma unroll
      for (int w = 0; w < E::kWords; ++w) {
        const uint32_t v = transpose_bytes(r.w[w], j);
        if (E::kBytes >= 4 || j < E::kBytes)
          *reinterpret_cast<uint32_t*>(p.codes + L::v_code(t0, E::kBytes * i + 4 * w + j)) = v;
      }
    }
  } else if (ok) {
    if constexpr (FMT == QL_KV_BF16) {
#pragma unroll
      for (int u = 0; u < E::N; ++u)
        *reinterpret_cast<uint16_t*>(p.codes + L::v_code(p.t, E::N * i + u)) =
            uint16_t(r.w[u / 2] >> (16 * (u & 1)));
    } else {
#pragma unroll
      for (int u = 0; u < E::kBytes; ++u)
        p.codes[L::v_code(p.t, E::kBytes * i + u)] = uint8_t(r.w[u / 4] >> (8 * (u & 3)));
    }
  }
  if (!ok) return;
  if constexpr (FMT == QL_KV_NVFP4) {
    constexpr int lanes = 16 / E::N;
    if (i % lanes == 0) p.scales[L::v_scale(p.t, i / lanes)] = uint8_t(r.scale);
  }
  if constexpr (FMT != QL_KV_BF16) {
    if (i == 0) p.scales[L::v_exp(p.t)] = uint8_t(r.exp);
  }
}

// --------------------------------------------------------------------------
// kv_append: a wave takes four tokens of one K or V head, 16 lanes a row, so
// that an aligned quad of V rows can be transposed in registers and stored as
// words (the layout keeps four tokens of an element together).  Bound by the
// bytes: 16384 tokens of 8 128-wide heads to 4 bits, 86 MB read and written in
// 23.4 us, 3.7 TB/s; a few tokens are one launch (3.4 us).
// --------------------------------------------------------------------------
template <int FMT, int D>
__global__ __launch_bounds__(64 * kWaves) void kv_append_kernel(
    KvGeom g, const void* k, const void* v, bool f32, int64_t tokens, int64_t k_stride,
    int64_t v_stride, const int64_t* slots) {
  constexpr int N = D / 16;
  const int lane = threadIdx.x & 63, i = lane & 15, j = lane >> 4;
  const int item = int(blockIdx.y) * kWaves + int(threadIdx.x >> 6);   // K heads, then V heads
  if (item >= 2 * g.n_kv) return;
  const bool is_v = item >= g.n_kv;
  const int head = is_v ? item - g.n_kv : item;
  const int64_t token = first_token(slots) + j;
  const int64_t slot = token >= 0 && token < tokens ? slots[token] : -1;
  const bool ok = slot_ok(g, slot);
  float x[N] = {};
  if (ok) {
    const void* from = is_v ? v : k;
    const int64_t off = token * (is_v ? v_stride : k_stride) + head * D + i * N;
    if (f32) load_row<true>(from, off, x);
    else load_row<false>(from, off, x);
  }
  const EncRow<FMT, D> r = encode_row<FMT, D>(x);
  const Place p = place_of<FMT, D>(g, ok ? slot : 0, head);
  if (is_v) {
    store_v<FMT, D>(p, i, j, whole_quad(slot, ok, j), ok, r);
  } else if (ok) {
    store_k<FMT, D>(p, i, r);
  }
}

// --------------------------------------------------------------------------
// qkv_norm_rope_append: a wave takes four tokens and a run of heads, whose
// rotation factors times weights it makes once; 16 lanes hold a row, so the sum
// of squares is four steps within them.  Bound by the bytes: 8192 tokens of 32
// query and 8 key heads of 128, bf16 in, 8-bit cache: 185 MB in 44.5 us,
// 4.1 TB/s; a few tokens are one launch (3.9 us).
// --------------------------------------------------------------------------
struct NormArgs {
  KvGeom g;
  const void* qkv;
  int64_t tokens;
  int64_t row_stride;
  int n_q;
  int heads_per_wave;
  const float* q_weight;
  const float* k_weight;
  float eps;
  const int32_t* positions;
  const float* rope;
  int64_t max_pos;
  int rot;
  void* q_out;
  const int64_t* slots;
};

// Rotations: half-split over the whole head (the partner is in another lane, at
// the same place), half-split over a part of it (or none; the partner may be
// anywhere: through LDS), pairs of neighbours.
enum { kRotWhole, kRotPart, kRotPairs };

template <int FMT, int D, int ROT, bool F32>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 2 : 4) void qkv_norm_rope_append_kernel(NormArgs a) {
  constexpr int N = D / 16;
  __shared__ float4 rows[ROT == kRotPart ? kWaves : 1][4][D / 4];   // each wave's rows
  const int lane = threadIdx.x & 63, i = lane & 15, j = lane >> 4, wave = threadIdx.x >> 6;
  const int64_t token = first_token(a.slots) + j;
  const bool in = token >= 0 && token < a.tokens;
  const int64_t slot = in ? a.slots[token] : -1;
  const bool ok = slot_ok(a.g, slot);
  const bool quad = whole_quad(slot, ok, j);
  const int heads = a.n_q + 2 * a.g.n_kv;
  const int half = a.rot >> 1;

  // Norm and rotation of element d, whose partner is pd, together:
  //   y[d] = r (x[d] w[d] c[d] +- x[pd] w[pd] s[d]),  r = rsqrt(mean(x^2) + eps);
  // wc and ws hold the factors of x[d] and x[pd] for the heads of one kind
  // (queries or keys) of this token.  Queries, which end in bf16, are computed
  // in binary32; keys, whose rounding to a code follows, in binary64, so that
  // the code is that of the exact value (binary32 errors move one code in 10^5
  // to its neighbour).  One head in six is a key's: 8192 tokens of 48 128-wide
  // heads take 46 us either way, 4000 of 84 64-wide ones 22 us against 18.
  auto factors = [&](const float* weight, auto& wc, auto& ws) {
    int64_t pos = in && half ? a.positions[token] : 0;
    pos = pos < 0 ? 0 : pos >= a.max_pos ? a.max_pos - 1 : pos;
    const float* t = half ? a.rope + pos * a.rot : nullptr;
#pragma unroll
    for (int u = 0; u < N; u += 4) {
      const int d = i * N + u;
      f32x4 w = {1, 1, 1, 1}, c = {1, 1, 1, 1}, s = {0, 0, 0, 0}, wp = {1, 1, 1, 1};
      if (weight) w = load4(weight + d);
      const int h = ROT == kRotWhole ? D / 2 : half;
      if (ROT == kRotPairs && d + 4 <= a.rot) {
        const f32x2 cv = load2(t + d / 2), sv = load2(t + half + d / 2);
        c = f32x4{cv[0], cv[0], cv[1], cv[1]}, s = f32x4{-sv[0], sv[0], -sv[1], sv[1]};
        wp = f32x4{w[1], w[0], w[3], w[2]};
      } else if (ROT == kRotWhole || (ROT == kRotPart && (d + 4 <= h || (d >= h && d + 4 <= a.rot)))) {
        const int at = d < h ? d : d - h;
        c = load4(t + at), s = load4(t + h + at);
        if (d < h) s = -s;
        if (weight) wp = load4(weight + (d < h ? d + h : at));
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int e = d + x;
          if (e >= a.rot) continue;
          const bool first = ROT == kRotPairs ? (x & 1) == 0 : e < half;
          const int at = ROT == kRotPairs ? e >> 1 : first ? e : e - half;
          c[x] = t[at];
          s[x] = first ? -t[half + at] : t[half + at];
          if (ROT == kRotPairs) wp[x] = w[x ^ 1];
          else if (weight) wp[x] = weight[first ? e + half : e - half];
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        typedef std::remove_reference_t<decltype(wc[0])> T;
        wc[u + x] = static_cast<T>(w[x]) * static_cast<T>(c[x]);
        ws[u + x] = static_cast<T>(wp[x]) * static_cast<T>(s[x]);
      }
    }
  };

  auto norm_rope = [&](const float (&x)[N], bool norm, const auto& wc, const auto& ws, auto& y) {
    typedef std::remove_const_t<std::remove_reference_t<decltype(wc[0])>> T;
    T r = 1;
    if (norm) {
      T sum = 0;
#pragma unroll
      for (int u = 0; u < N; ++u) sum = fma_of(static_cast<T>(x[u]), static_cast<T>(x[u]), sum);
      r = rsqrt_of(fma_of(row_sum(sum), static_cast<T>(1.0f / D), static_cast<T>(a.eps)));
    }
    // Elements from rot on have none: -0 times their factor 0 adds -0, which
    // leaves every value as it is, an infinity and a -0 as well.
    float partner[N];
    if constexpr (ROT == kRotPairs) {
#pragma unroll
      for (int u = 0; u < N; ++u) partner[u] = i * N + u < a.rot ? x[u ^ 1] : -0.0f;
    } else if constexpr (ROT == kRotWhole) {
      // half a row on is 8 of its 16 lanes on
#pragma unroll
      for (int u = 0; u < N; ++u) partner[u] = dpp<0x128>(x[u]);
    } else {
      // the wave's own rows: its LDS accesses run in order, the fences keep
      // the compiler from moving them past each other
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < N; u += 4)
        rows[wave][j][(i * N + u) / 4] = make_float4(x[u], x[u + 1], x[u + 2], x[u + 3]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const float* row = reinterpret_cast<const float*>(rows[wave][j]);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int d = i * N + u;
        const float other = row[d < half ? d + half : d < a.rot ? d - half : d];
        partner[u] = d < a.rot ? other : -0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
      y[u] = fma_of(static_cast<T>(partner[u]), ws[u], x[u] * wc[u]) * r;
  };

  // A loop of its own for each kind of head: with one of three kinds of stores
  // behind a branch, the compiler would wait for all of them before the next
  // row.  The row after the one worked on is under way.
  const int first = (int(blockIdx.y) * kWaves + wave) * a.heads_per_wave;
  const int end = first + a.heads_per_wave < heads ? first + a.heads_per_wave : heads;
  auto sweep = [&](int from, int to, auto&& work) {
    from = from > first ? from : first;
    to = to < end ? to : end;
    if (from >= to) return;
    const int64_t off = token * a.row_stride + i * N;
    float next[N] = {};
    if (in) load_row<F32>(a.qkv, off + int64_t(from) * D, next);
    for (int h = from; h < to; ++h) {
      float x[N];
#pragma unroll
      for (int u = 0; u < N; ++u) x[u] = next[u];
      if (in && h + 1 < to) load_row<F32>(a.qkv, off + int64_t(h + 1) * D, next);
      work(h, x);
    }
  };
  const int k0 = a.n_q, v0 = a.n_q + a.g.n_kv;
  float qc[N], qs[N];
  if (first < k0) factors(a.q_weight, qc, qs);
  sweep(0, k0, [&](int h, float (&x)[N]) {
    float y[N];
    norm_rope(x, a.q_weight != nullptr, qc, qs, y);
    if (in) store_row_bf16(a.q_out, (token * a.n_q + h) * D + i * N, y);
  });
  double kc[N], ks[N];
  if (end > k0 && first < v0) factors(a.k_weight, kc, ks);
  sweep(k0, v0, [&](int h, float (&x)[N]) {
    double y[N];
    norm_rope(x, a.k_weight != nullptr, kc, ks, y);
    const EncRow<FMT, D> r = encode_row<FMT, D>(y);
    if (ok) store_k<FMT, D>(place_of<FMT, D>(a.g, slot, h - k0), i, r);
  });
  sweep(v0, heads, [&](int h, float (&x)[N]) {
    const EncRow<FMT, D> r = encode_row<FMT, D>(x);
    store_v<FMT, D>(place_of<FMT, D>(a.g, ok ? slot : 0, h - v0), i, j, quad, ok, r);
  });
}

// --------------------------------------------------------------------------
// kv_gather: as kv_append the other way (16384 tokens of 8 128-wide heads from 4
// bits: 86 MB in 18.9 us, 4.5 TB/s).
// --------------------------------------------------------------------------
template <int FMT, int D>
__device__ __forceinline__ void decode_row(const EncRow<FMT, D>& r, float (&x)[D / 16]) {
  constexpr int N = D / 16;
  if constexpr (FMT == QL_KV_BF16) {
#pragma unroll
    for (int u = 0; u < N; ++u)
      x[u] = __uint_as_float(u & 1 ? r.w[u / 2] & 0xFFFF0000u : r.w[u / 2] << 16);
  } else {
    const float p = __uint_as_float(r.exp << 23);
    if constexpr (FMT == QL_KV_E4M3) {
#pragma unroll
      for (int u = 0; u < N; u += 2) {
        const f32x2 v = u & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8(int(r.w[u / 4]), true)
                              : __builtin_amdgcn_cvt_pk_f32_fp8(int(r.w[u / 4]), false);
        x[u] = v[0] * p, x[u + 1] = v[1] * p;
      }
    } else {
      const float sv = __builtin_amdgcn_cvt_f32_fp8(int(r.scale), 0);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        f32x2 v;
        switch (i & 3) {
          case 0: v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.w[i / 4], 1.0f, 0); break;
          case 1: v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.w[i / 4], 1.0f, 1); break;
          case 2: v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.w[i / 4], 1.0f, 2); break;
          default: v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.w[i / 4], 1.0f, 3); break;
        }
        x[2 * i] = v[0] * sv * p, x[2 * i + 1] = v[1] * sv * p;
      }
    }
  }
}

template <int FMT, int D>
__device__ __forceinline__ void load_k(const Place& p, int i, EncRow<FMT, D>& r) {
  using L = KvLayout<FMT, D>;
  using E = EncRow<FMT, D>;
  if constexpr (E::kBytes == 2) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p.codes + L::k_code(p.t, 2 * i));
  } else {
    constexpr int piece = E::kBytes < 16 ? E::kBytes : 16;
#pragma unroll
    for (int c = 0; c < E::kBytes / piece; ++c) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(
          p.codes + L::k_code(p.t, E::kBytes * i + piece * c));
#pragma unroll
      for (int w = 0; w < piece / 4; ++w) r.w[c * (piece / 4) + w] = q[w];
    }
  }
  if constexpr (FMT == QL_KV_NVFP4) r.scale = p.scales[L::k_scale(p.t, i * E::N / 16)];
  if constexpr (FMT != QL_KV_BF16) r.exp = p.scales[L::k_exp(p.t)];
}

// V: the four tokens of a quad lie side by side, so a lane reads its elements
// of all four in wide loads and keeps its own token's.
template <int FMT, int D>
__device__ __forceinline__ void load_v(const Place& p, int i, int j, bool quad, EncRow<FMT, D>& r) {
  using L = KvLayout<FMT, D>;
  using E = EncRow<FMT, D>;
  if constexpr (FMT == QL_KV_BF16) {
    // 8192 tokens of 8 128-wide heads: 14.3 us this way, 27.2 the other
    if (quad) {
#pragma unroll
      for (int w = 0; w < E::kWords / 2; ++w) {
        const uint2 v = *reinterpret_cast<const uint2*>(
            p.codes + L::v_code(p.t & ~3, E::N * i + 4 * w + j));
        const uint2 o = transpose_halves(v.x, v.y, j);
        r.w[2 * w] = o.x, r.w[2 * w + 1] = o.y;
      }
      return;
    }
  }
  constexpr int units = FMT == QL_KV_BF16 ? E::N : E::kBytes;      // elements, codes or pairs
  constexpr int words = FMT == QL_KV_BF16 ? 2 * units : units;
  constexpr int wide = words < 4 ? words : 4;
  uint32_t q[words];
#pragma unroll
  for (int w = 0; w < words; w += wide) {
    typedef uint32_t Wide __attribute__((ext_vector_type(wide)));
    const Wide v = reinterpret_cast<const Wide*>(p.codes + L::v_code(p.t & ~3, units * i))[w / wide];
#pragma unroll
    for (int x = 0; x < wide; ++x) q[w + x] = v[x];
  }
#pragma unroll
  for (int w = 0; w < E::kWords; ++w) {
    if constexpr (FMT == QL_KV_BF16) {
      const int sh = 16 * (p.t & 1);
      const uint32_t a = p.t & 2 ? q[4 * w + 1] : q[4 * w], b = p.t & 2 ? q[4 * w + 3] : q[4 * w + 2];
      r.w[w] = (a >> sh & 0xFFFFu) | (b >> sh) << 16;
    } else {
      const uint32_t sel = uint32_t(p.t & 3) | uint32_t(4 + (p.t & 3)) << 8 | 0x0C0C0000u;
      const uint32_t lo = __builtin_amdgcn_perm(q[4 * w + 1 < words ? 4 * w + 1 : 0], q[4 * w], sel);
      r.w[w] = lo;
      if constexpr (words >= 4)
        r.w[w] = lo | __builtin_amdgcn_perm(q[4 * w + 3], q[4 * w + 2], sel) << 16;
    }
  }
  if constexpr (FMT == QL_KV_NVFP4) r.scale = p.scales[L::v_scale(p.t, i * E::N / 16)];
  if constexpr (FMT != QL_KV_BF16) r.exp = p.scales[L::v_exp(p.t)];
}

template <int FMT, int D>
__global__ __launch_bounds__(64 * kWaves) void kv_gather_kernel(KvGeom g, const int64_t* slots,
                                                                int64_t tokens, void* k, void* v,
                                                                bool f32) {
  constexpr int N = D / 16;
  const int lane = threadIdx.x & 63, i = lane & 15, j = lane >> 4;
  const int item = int(blockIdx.y) * kWaves + int(threadIdx.x >> 6);
  if (item >= 2 * g.n_kv) return;
  const bool is_v = item >= g.n_kv;
  const int head = is_v ? item - g.n_kv : item;
  const int64_t token = int64_t(blockIdx.x) * 4 + j;
  const int64_t slot = token < tokens ? slots[token] : -1;
  const bool ok = slot_ok(g, slot);
  const Place p = place_of<FMT, D>(g, ok ? slot : 0, head);
  EncRow<FMT, D> r = {};
  const bool quad = whole_quad(slot, ok, j);
  float x[N] = {};
  if (ok) {
    if (is_v) load_v<FMT, D>(p, i, j, quad, r);
    else load_k<FMT, D>(p, i, r);
    decode_row<FMT, D>(r, x);
  }
  if (token >= tokens) return;
  void* out = is_v ? v : k;
  const int64_t off = (token * g.n_kv + head) * D + i * N;
  if (f32) {
    float* o = static_cast<float*>(out) + off;
#pragma unroll
    for (int u = 0; u < N; u += 4)
      *reinterpret_cast<float4*>(o + u) = make_float4(x[u], x[u + 1], x[u + 2], x[u + 3]);
  } else {
    store_row_bf16(out, off, x);
  }
}

// --------------------------------------------------------------------------
// kv_commit: one block per sequence, kv head and half (K or V).  Source and
// target rows of a sequence overlap, so every row is read into LDS before
// the first is written.
// --------------------------------------------------------------------------
constexpr int kMaxPath = 64;

template <int FMT, int D>
__global__ __launch_bounds__(256) void kv_commit_kernel(KvGeom g, const int32_t* cu_q,
                                                        const int32_t* kv_lens,
                                                        const int32_t* table, int64_t table_stride,
                                                        int64_t table_cols, const int32_t* path,
                                                        int max_path) {
  using L = KvLayout<FMT, D>;
  constexpr int kGroups = FMT == QL_KV_NVFP4 ? D / 16 : 0;
  constexpr int kUnit = FMT == QL_KV_BF16 ? 2 : 1;     // bytes that stay together in V
  __shared__ __align__(16) uint8_t codes[kMaxPath][L::kRow];
  __shared__ uint8_t scales[kMaxPath][kGroups + 1];
  __shared__ Place from[kMaxPath], to[kMaxPath];       // of the rows that move
  __shared__ int moves;
  const int head = blockIdx.x, tid = threadIdx.x;
  const bool is_v = blockIdx.y != 0;
  const int64_t b = blockIdx.z;
  const int64_t nodes = cu_q[b + 1] - cu_q[b], len = kv_lens[b];
  const int64_t ctx = len > nodes ? len - nodes : 0;
  if (tid < 64) {
    auto slot_at = [&](int64_t pos) -> int64_t {
      const int64_t col = pos >> g.page_shift;
      if (col >= table_cols) return -1;
      const int64_t page = table[b * table_stride + col];
      if (page < 0 || page >= g.n_pages) return -1;
      return (page << g.page_shift) + (pos & ((int64_t(1) << g.page_shift) - 1));
    };
    const int64_t node = tid < max_path ? path[b * max_path + tid] : -1;
    int64_t s = -1, d = -1;
    if (node >= 0 && node < nodes && ctx + node < len && node != tid && ctx + tid < len) {
      s = slot_at(ctx + node);
      d = slot_at(ctx + tid);
    }
    const uint64_t some = __ballot(s >= 0 && d >= 0);
    if (some >> tid & 1) {
      const int at = __popcll(some & ((uint64_t(1) << tid) - 1));
      from[at] = place_of<FMT, D>(g, s, head);
      to[at] = place_of<FMT, D>(g, d, head);
    }
    if (tid == 0) moves = __popcll(some);
  }
  __syncthreads();

  const int count = moves;
  auto rows = [&](const Place* places, auto&& move) {
    if (!is_v) {
      constexpr int chunks = L::kRow / L::kLoad;
      for (int u = tid; u < count * chunks; u += 256) {
        const int n = u / chunks, c = u % chunks;
        const Place p = places[n];
        if constexpr (L::kLoad == 16)
          move(reinterpret_cast<uint4*>(p.codes + L::k_code(p.t, 16 * c)),
               reinterpret_cast<uint4*>(codes[n] + 16 * c));
        else
          move(reinterpret_cast<uint2*>(p.codes + L::k_code(p.t, 8 * c)),
               reinterpret_cast<uint2*>(codes[n] + 8 * c));
      }
    } else {
      constexpr int units = L::kRow / kUnit;
      for (int u = tid; u < count * units; u += 256) {
        const int n = u / units, c = u % units;
        const Place p = places[n];
        if constexpr (kUnit == 2)
          move(reinterpret_cast<uint16_t*>(p.codes + L::v_code(p.t, c)),
               reinterpret_cast<uint16_t*>(codes[n] + 2 * c));
        else
          move(p.codes + L::v_code(p.t, c), codes[n] + c);
      }
    }
    if constexpr (FMT != QL_KV_BF16) {
      for (int u = tid; u < count * (kGroups + 1); u += 256) {
        const int n = u / (kGroups + 1), c = u % (kGroups + 1);
        const Place p = places[n];
        const int off = c == kGroups ? (is_v ? L::v_exp(p.t) : L::k_exp(p.t))
                                     : (is_v ? L::v_scale(p.t, c) : L::k_scale(p.t, c));
        move(p.scales + off, &scales[n][c]);
      }
    }
  };
  rows(from, [](auto* cache, auto* lds) { *lds = *cache; });
  __syncthreads();
  rows(to, [](auto* cache, auto* lds) { *cache = *lds; });
}

}  // namespace

// A grid has less than 2^32 threads along x, so more tokens than this take
// several launches: calls launch(first, count).
template <typename F>
static hipError_t by_launch(int64_t tokens, F&& launch) {
  constexpr int64_t most = int64_t(1) << 25;
  for (int64_t t = 0; t < tokens; t += most) {
    launch(t, tokens - t < most ? tokens - t : most);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
// `rows` rows on from p.
static const void* ahead(const void* p, int64_t rows, int64_t stride, int dtype) {
  return static_cast<const uint8_t*>(p) + rows * stride * (dtype == QL_F32 ? 4 : 2);
}
static void* ahead(void* p, int64_t rows, int64_t stride, int dtype) {
  return static_cast<uint8_t*>(p) + rows * stride * (dtype == QL_F32 ? 4 : 2);
}

hipError_t launch_kv_append(const KvGeom& g, int fmt, int d, const void* k, const void* v,
                            int x_dtype, int64_t tokens, int64_t k_stride, int64_t v_stride,
                            const int64_t* slots, hipStream_t s) {
  return kv_dispatch(fmt, d, [&](auto f, auto n) {
    return by_launch(tokens, [&](int64_t t, int64_t count) {
      const dim3 grid(quads(count), unsigned((2 * g.n_kv + kWaves - 1) / kWaves));
      kv_append_kernel<decltype(f)::value, decltype(n)::value><<<grid, 64 * kWaves, 0, s>>>(
          g, ahead(k, t, k_stride, x_dtype), ahead(v, t, v_stride, x_dtype), x_dtype == QL_F32,
          count, k_stride, v_stride, slots + t);
    });
  });
}

hipError_t launch_qkv_norm_rope_append(const KvGeom& g, int fmt, int d, const void* qkv,
                                       int x_dtype, int64_t tokens, int64_t row_stride, int n_q,
                                       const float* q_weight, const float* k_weight, float eps,
                                       const int32_t* positions, const float* rope,
                                       int64_t max_pos, int rot, bool interleaved, void* q_out,
                                       const int64_t* slots, hipStream_t s) {
  const int heads = n_q + 2 * g.n_kv;
  // Heads per wave: a wave's cosines and sines are read once for all of its
  // heads, but there should be waves enough: 8192, or 4096 of the longest rows
  // (2000 tokens of 28 256-wide heads: 16.3 us with 4096, 20.4 with 8192; 4000
  // of 84 64-wide ones 20.7 and 17.7).
  const int64_t waves = (tokens + 3) / 4 * heads, full = d == 256 ? 4096 : 8192;
  const int most = (heads + kWaves - 1) / kWaves;
  const int hpw = waves <= full ? 1 : waves / full < most ? int(waves / full) : most;
  return kv_dispatch(fmt, d, [&](auto f, auto n) {
    constexpr int FMT = decltype(f)::value, D = decltype(n)::value;
    auto go = [&](auto rot_c, auto f32_c) {
      return by_launch(tokens, [&](int64_t t, int64_t count) {
        const NormArgs a{g, ahead(qkv, t, row_stride, x_dtype), count, row_stride, n_q, hpw,
                         q_weight, k_weight, eps, positions ? positions + t : nullptr, rope,
                         max_pos, rot, ahead(q_out, t, int64_t(n_q) * d, QL_BF16), slots + t};
        const dim3 grid(quads(count), unsigned((heads + kWaves * hpw - 1) / (kWaves * hpw)));
        qkv_norm_rope_append_kernel<FMT, D, decltype(rot_c)::value, decltype(f32_c)::value>
            <<<grid, 64 * kWaves, 0, s>>>(a);
      });
    };
    auto by_type = [&](auto rot_c) {
      return x_dtype == QL_F32 ? go(rot_c, std::true_type{}) : go(rot_c, std::false_type{});
    };
    return interleaved ? by_type(std::integral_constant<int, kRotPairs>{})
           : rot == D  ? by_type(std::integral_constant<int, kRotWhole>{})
                       : by_type(std::integral_constant<int, kRotPart>{});
  });
}

hipError_t launch_kv_gather(const KvGeom& g, int fmt, int d, const int64_t* slots, int64_t tokens,
                            void* k, void* v, int y_dtype, hipStream_t s) {
  const int64_t row = int64_t(g.n_kv) * d;
  return kv_dispatch(fmt, d, [&](auto f, auto n) {
    return by_launch(tokens, [&](int64_t t, int64_t count) {
      const dim3 grid(unsigned((count + 3) / 4), unsigned((2 * g.n_kv + kWaves - 1) / kWaves));
      kv_gather_kernel<decltype(f)::value, decltype(n)::value><<<grid, 64 * kWaves, 0, s>>>(
          g, slots + t, count, ahead(k, t, row, y_dtype), ahead(v, t, row, y_dtype),
          y_dtype == QL_F32);
    });
  });
}

hipError_t launch_kv_commit(const KvGeom& g, int fmt, int d, int64_t n_seqs, const int32_t* cu_q,
                            const int32_t* kv_lens, const int32_t* table, int64_t table_stride,
                            int64_t table_cols, const int32_t* path, int max_path, hipStream_t s) {
  const dim3 grid(unsigned(g.n_kv), 2, unsigned(n_seqs));
  return kv_dispatch(fmt, d, [&](auto f, auto n) {
    kv_commit_kernel<decltype(f)::value, decltype(n)::value><<<grid, 256, 0, s>>>(
        g, cu_q, kv_lens, table, table_stride, table_cols, path, max_path);
    return hipGetLastError();
  });
}

}  // namespace qlin
