// Layout of the paged key/value cache and the checks its entry points share.
// Internal; the public description is in include/qlin.h.
#pragma once

#include "../../include/qlin.h"
#include "qlin_internal.hpp"

#include <type_traits>

namespace qlin {

// A block is 16 tokens of one kv head.  Codes of every block come first
// ([n_pages][n_kv][page_size / 16] blocks of K codes then V codes), the
// scales of every block after them in the same order.  The codes of a block
// are laid out in the order the attention kernel's matrix operands take them:
// one wave load of a block (lane l, load i) reads kLoad bytes at
// (64 i + l) kLoad, and those are
//   K: token l % 16, elements of chunk c = 4 i + l / 16 (kLoad bytes of a row)
//   V: tokens 4 (l / 16) .. + 3, the element range kDC (l % 16) .. + kDC - 1
//      of segment i (16 kDC elements), the four tokens of one element (one
//      pair of elements for 4-bit codes) side by side.
// So a wave reads whole contiguous blocks, and every operand register is
// made from registers of the same lane.
template <int FMT, int D>
struct KvLayout {
  static constexpr int kRow = FMT == QL_KV_BF16 ? 2 * D : FMT == QL_KV_E4M3 ? D : D / 2;
  static constexpr int kCodes = 32 * kRow;     // bytes of a block's K and V codes
  static constexpr int kScales = FMT == QL_KV_BF16 ? 0 : FMT == QL_KV_E4M3 ? 32 : 2 * D + 32;
  static constexpr int kLoad = kRow / 4 < 16 ? kRow / 4 : 16;  // bytes per lane and load
  static constexpr int kLoads = kRow / 4 / kLoad;              // loads of K (or V) per block
  static constexpr int kEC = FMT == QL_KV_BF16 ? kLoad / 2     // elements of a K chunk
                             : FMT == QL_KV_E4M3 ? kLoad : 2 * kLoad;
  static constexpr int kDC = kEC / 4;                          // elements of V per lane and load
  static constexpr int kGPC = kEC / 16;        // NVFP4 groups per K chunk (1 or 2)
  static constexpr int kExp = FMT == QL_KV_NVFP4 ? 2 * D : 0;  // row exponents in the scales

  // Byte offsets in a block's codes / scales.
  __host__ __device__ static constexpr int k_code(int t, int b) {   // byte b of token t's row
    return (b / kLoad) * (16 * kLoad) + t * kLoad + b % kLoad;
  }
  // V: element d (BF16: byte offset of the element; E4M3: its byte), or pair
  // d (NVFP4) of token t
  __host__ __device__ static constexpr int v_code(int t, int u) {
    constexpr int seg = FMT == QL_KV_NVFP4 ? 8 * kDC : 16 * kDC;   // units per segment
    constexpr int size = FMT == QL_KV_BF16 ? 2 : 1;
    return 16 * kRow + size * ((u / seg) * (16 * seg) + (t / 4) * (4 * seg) + (u % seg) * 4 + t % 4);
  }
  __host__ __device__ static constexpr int k_scale(int t, int g) {
    constexpr int per = kGPC > 0 ? kGPC : 1;
    return (g / per) * (16 * per) + t * per + g % per;
  }
  __host__ __device__ static constexpr int v_scale(int t, int g) { return D + g * 16 + t; }
  __host__ __device__ static constexpr int k_exp(int t) { return kExp + (t / 4) * 8 + t % 4; }
  __host__ __device__ static constexpr int v_exp(int t) { return k_exp(t) + 4; }
};

// Smallest stored row exponent (e + 127): a row's scale is 2^e, e >= -100.
constexpr int kKvExpMin = 27;

// Geometry of a cache, passed to the kernels by value.
struct KvGeom {
  uint8_t* codes;
  uint8_t* scales;
  int64_t n_pages;
  int n_kv;
  int page_shift;       // log2(page_size)
};

inline int kv_row_bytes(int fmt, int64_t d) {
  return int(fmt == QL_KV_BF16 ? 2 * d : fmt == QL_KV_E4M3 ? d : d / 2);
}
inline int kv_scale_bytes(int fmt, int64_t d) {
  return int(fmt == QL_KV_BF16 ? 0 : fmt == QL_KV_E4M3 ? 32 : 2 * d + 32);
}

// Block index of (page, kv head, block of the page).
__device__ __forceinline__ int64_t kv_block(const KvGeom& g, int64_t page, int head, int bip) {
  return ((page * g.n_kv + head) << (g.page_shift - 4)) + bip;
}

// Calls f(format, head size) with both as integral constants.
template <typename F>
hipError_t kv_dispatch(int fmt, int d, F&& f) {
  auto by_d = [&](auto fmt_c) -> hipError_t {
    switch (d) {
      case 64: return f(fmt_c, std::integral_constant<int, 64>{});
      case 128: return f(fmt_c, std::integral_constant<int, 128>{});
      case 256: return f(fmt_c, std::integral_constant<int, 256>{});
      default: return hipErrorInvalidValue;
    }
  };
  switch (fmt) {
    case QL_KV_BF16: return by_d(std::integral_constant<int, QL_KV_BF16>{});
    case QL_KV_E4M3: return by_d(std::integral_constant<int, QL_KV_E4M3>{});
    case QL_KV_NVFP4: return by_d(std::integral_constant<int, QL_KV_NVFP4>{});
    default: return hipErrorInvalidValue;
  }
}

// Launchers (validated arguments).
hipError_t launch_kv_append(const KvGeom& g, int fmt, int d, const void* k, const void* v,
                            int x_dtype, int64_t tokens, int64_t k_stride, int64_t v_stride,
                            const int64_t* slots, hipStream_t s);
hipError_t launch_qkv_norm_rope_append(const KvGeom& g, int fmt, int d, const void* qkv,
                                       int x_dtype, int64_t tokens, int64_t row_stride, int n_q,
                                       const float* q_weight, const float* k_weight, float eps,
                                       const int32_t* positions, const float* rope,
                                       int64_t max_pos, int rot, bool interleaved, void* q_out,
                                       const int64_t* slots, hipStream_t s);
hipError_t launch_kv_gather(const KvGeom& g, int fmt, int d, const int64_t* slots, int64_t tokens,
                            void* k, void* v, int y_dtype, hipStream_t s);
hipError_t launch_kv_commit(const KvGeom& g, int fmt, int d, int64_t n_seqs, const int32_t* cu_q,
                            const int32_t* kv_lens, const int32_t* table, int64_t table_stride,
                            int64_t table_cols, const int32_t* path, int max_path, hipStream_t s);

struct KvAttnArgs {
  KvGeom g;
  const void* q;          // bf16 [tokens, n_q, d], token stride q_stride elements
  int64_t q_stride;
  int64_t tokens;
  int n_seqs;
  int n_q;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  const int32_t* table;
  int64_t table_stride;
  int64_t table_cols;
  int max_q;
  int64_t max_kv;
  const uint64_t* tree;
  float scale;
  void* y;                // bf16 [tokens, n_q, d]
  float* part_o;          // [parts][max_q * n_q][d]
  float* part_ml;         // [parts][max_q * n_q][2]
  int32_t* first;         // [n_seqs + 1]: each sequence's first part
  int parts;              // parts of the keys of all sequences; n_seqs: none is split
  int units;              // parts * n_kv
  int row_blocks;
};
struct KvAttnPlan {
  int rows;               // query rows per block: 16 (narrow), 32 (pair), 64 (wide)
  int64_t row_blocks;
  int64_t parts;
};
KvAttnPlan kv_attention_plan(int fmt, int d, int n_q, int n_kv, int64_t n_seqs, int64_t max_q,
                             int64_t max_kv);
size_t kv_attention_ws_bytes(const KvAttnPlan& p, int64_t n_seqs, int64_t max_q, int n_q, int d);
hipError_t launch_kv_attention(int fmt, int d, const KvAttnPlan& p, KvAttnArgs a, hipStream_t s);

}  // namespace qlin
