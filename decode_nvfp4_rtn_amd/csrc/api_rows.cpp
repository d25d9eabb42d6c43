// extern "C" entry points of the layers whose rows choose their own weights:
// argument validation and dispatch.  As in api.cpp every check runs on the host
// before any device work.  See include/qlin.h for the contract.
#include "../../include/qlin.h"
#include "moe.hpp"

using namespace qlin;

namespace {

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool aligned16(const void* p) { return aligned(p, 16); }

int launch_status(hipError_t e) { return e == hipSuccess ? QL_OK : QL_EHIP; }

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t kMostRows = (int64_t(1) << 24) - 1;   // a launch has fewer than 2^32 threads
constexpr int64_t kMostTopK = 64;
constexpr int64_t kMostSpan = int64_t(1) << 47;          // bytes of strided rows: no address space has more

bool dtype_ok(int d) { return d == QL_F32 || d == QL_BF16; }

bool groups_ok(int64_t groups) { return groups >= 1 && groups <= kMostGroups; }

// A plan's workspace: `need` bytes of it.
int check_workspace(size_t need, const void* workspace, size_t bytes) {
  if (!need) return QL_OK;
  if (!workspace) return QL_EINVAL;
  if (!aligned16(workspace)) return QL_EALIGN;
  return bytes < need ? QL_EWORKSPACE : QL_OK;
}

// Sizes shared by the two products; -1 if there is work, a status otherwise.
int check_product(int64_t pairs, int64_t top_k, int64_t n_experts, int64_t expert_bytes, int fmt,
                  int64_t n, int64_t k, unsigned flags, int y_dtype) {
  if (pairs < 0 || n < 0 || k < 0 || (flags & ~(QL_ROWS_GATHER | QL_ROWS_SILU_MUL))) return QL_EINVAL;
  if (!dtype_ok(y_dtype)) return QL_EDTYPE;
  if (!groups_ok(n_experts) || top_k < 1 || top_k > kMostTopK || pairs > kMostRows) return QL_ESHAPE;
  if (pairs % top_k) return QL_ESHAPE;
  if (n == 0 || k == 0 || k % 128 || n % (flags & QL_ROWS_SILU_MUL ? 32 : 16)) return QL_ESHAPE;
  if (n > (int64_t(1) << 24) || k > (int64_t(1) << 20) || n * k > (int64_t(1) << 31)) return QL_ESHAPE;
  if (pairs == 0) return QL_OK;
  if (expert_bytes % 16) return QL_EALIGN;
  if (expert_bytes < int64_t(repack_weights_bytes(fmt, n, k)) || expert_bytes > (int64_t(1) << 40))
    return QL_EWORKSPACE;
  return -1;
}

// Rows of `width` bytes, `stride` bytes apart, that a call reads or writes.
struct Rows {
  const void* at;
  int64_t count, stride, width;
};

// Whether two sets of rows share bytes.  Rows of one stride may lie side by side
// (slices of a fused projection); of two strides, where one set lies within the
// other's, they count as shared.
bool overlap(const Rows& a, const Rows& b) {
  const uint64_t at = reinterpret_cast<uintptr_t>(a.at), bt = reinterpret_cast<uintptr_t>(b.at);
  const uint64_t a_all = uint64_t((a.count - 1) * a.stride + a.width);
  const uint64_t b_all = uint64_t((b.count - 1) * b.stride + b.width);
  if (bt >= at ? bt - at >= a_all : at - bt >= b_all) return false;
  if (a.stride != b.stride) return true;
  const uint64_t s = uint64_t(a.stride);
  const uint64_t b_past = bt >= at ? (bt - at) % s : (s - (at - bt) % s) % s;   // b's column in a's rows
  return b_past < uint64_t(a.width) || b_past + uint64_t(b.width) > s;
}

Rows whole(const void* at, int64_t rows, int64_t width) { return Rows{at, rows, width, width}; }

int64_t bytes_of(int dtype) { return dtype == QL_F32 ? 4 : 2; }

// Whether a plan's arrays share bytes with what the plan is made from.
bool plan_over(const Rows& from, const int32_t* order, const int32_t* where, const int32_t* offsets,
               int64_t rows, int64_t groups) {
  return overlap(whole(order, 1, 4 * rows), from) || overlap(whole(where, 1, 4 * rows), from) ||
         overlap(whole(offsets, 1, 4 * (groups + 1)), from);
}

// The rows that a product writes.
Rows written(int64_t pairs, int64_t n, unsigned flags, const void* y, int y_dtype) {
  return whole(y, pairs, (flags & QL_ROWS_SILU_MUL ? n / 2 : n) * bytes_of(y_dtype));
}

MoeGemm product(const void* experts, int64_t n_experts, int64_t expert_bytes, const int32_t* order,
                const int32_t* offsets, int64_t pairs, int64_t top_k, int64_t n, int64_t k,
                unsigned flags, void* y, int y_dtype) {
  MoeGemm g{};
  g.plan = RowPlan{order, offsets, int(n_experts), int(pairs)};
  g.top_k = int(top_k);
  g.gather = (flags & QL_ROWS_GATHER) != 0;
  g.silu_mul = (flags & QL_ROWS_SILU_MUL) != 0;
  g.experts = static_cast<const uint8_t*>(experts);
  g.blob_stride = expert_bytes;
  g.n = int(n);
  g.k = int(k);
  g.y = y;
  g.y_dtype = y_dtype;
  return g;
}

}  // namespace

extern "C" {

size_t group_rows_workspace(int64_t rows, int64_t groups) {
  if (rows < 0 || rows > kMostRows || !groups_ok(groups)) return 0;
  return group_rows_ws_bytes(rows, 1, groups);
}

int group_rows(const int32_t* ids, int64_t rows, int64_t groups, int32_t* order, int32_t* where,
               int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream) {
  if (rows < 0) return QL_EINVAL;
  if (rows > kMostRows || !groups_ok(groups)) return QL_ESHAPE;
  if (!offsets || (rows && (!ids || !order || !where))) return QL_EINVAL;
  if (!aligned(ids, 4) || !aligned(order, 4) || !aligned(where, 4) || !aligned(offsets, 4)) return QL_EALIGN;
  const int st = check_workspace(group_rows_workspace(rows, groups), workspace, workspace_bytes);
  if (st != QL_OK) return st;
  if (rows && plan_over(whole(ids, 1, 4 * rows), order, where, offsets, rows, groups)) return QL_EINVAL;
  return launch_status(launch_group_rows(ids, rows, int(groups), order, where, offsets,
                                         static_cast<int32_t*>(workspace), as_stream(stream)));
}

size_t moe_route_workspace(int64_t tokens, int64_t experts, int64_t top_k) {
  if (tokens < 0 || !groups_ok(experts) || top_k < 1 || top_k > kMostTopK || tokens > kMostRows / top_k)
    return 0;
  return group_rows_ws_bytes(tokens * top_k, top_k, experts);
}

int moe_route(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t row_stride,
              int64_t top_k, unsigned flags, int32_t* ids, float* weights, int32_t* order,
              int32_t* where, int32_t* offsets, void* workspace, size_t workspace_bytes,
              void* stream) {
  if (tokens < 0 || (flags & ~QL_ROUTE_RENORMALIZE)) return QL_EINVAL;
  if (!dtype_ok(dtype)) return QL_EDTYPE;
  if (!groups_ok(experts) || top_k < 1 || top_k > kMostTopK || top_k > experts || tokens > kMostRows / top_k)
    return QL_ESHAPE;
  if (row_stride < experts || row_stride > (int64_t(1) << 31)) return QL_ESHAPE;
  if (!offsets || (tokens && (!logits || !ids || !weights || !order || !where))) return QL_EINVAL;
  if (!aligned(logits, dtype == QL_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(order, 4) || !aligned(where, 4) || !aligned(offsets, 4))
    return QL_EALIGN;
  const int st = check_workspace(moe_route_workspace(tokens, experts, top_k), workspace, workspace_bytes);
  if (st != QL_OK) return st;
  if (tokens) {
    const int64_t size = bytes_of(dtype), pairs = tokens * top_k;
    const Rows from{logits, tokens, row_stride * size, experts * size};
    if (overlap(whole(ids, 1, 4 * pairs), from) || overlap(whole(weights, 1, 4 * pairs), from) ||
        plan_over(from, order, where, offsets, pairs, experts))
      return QL_EINVAL;
  }
  return launch_status(launch_moe_route(logits, dtype, tokens, int(experts), row_stride, int(top_k),
                                        (flags & QL_ROUTE_RENORMALIZE) != 0, ids, weights, order, where,
                                        offsets, static_cast<int32_t*>(workspace), as_stream(stream)));
}

int moe_gemm_w4a16(const void* x_bf16, const void* experts, int64_t n_experts, int64_t expert_bytes,
                   const int32_t* order, const int32_t* offsets, int64_t pairs, int64_t top_k,
                   int64_t n, int64_t k, unsigned flags, void* y, int y_dtype, void* stream) {
  const int st = check_product(pairs, top_k, n_experts, expert_bytes, QL_INT4_G128, n, k, flags, y_dtype);
  if (st >= QL_OK) return st;
  // at most a block of 1024 threads for each 32 places and 512 rows of the weights
  if (most_tiles(pairs, n_experts, 32) * ((n + 511) / 512) >= int64_t(1) << 22) return QL_ESHAPE;
  if (!x_bf16 || !experts || !offsets || !y || (!order && (flags & QL_ROWS_GATHER))) return QL_EINVAL;
  if (!aligned16(x_bf16) || !aligned16(experts) || !aligned16(y) || !aligned(order, 4) || !aligned(offsets, 4))
    return QL_EALIGN;
  const int64_t rows = flags & QL_ROWS_GATHER ? pairs / top_k : pairs;
  if (overlap(written(pairs, n, flags, y, y_dtype), whole(x_bf16, rows, 2 * k))) return QL_EINVAL;
  return launch_status(launch_moe_gemm_w4a16(
      product(experts, n_experts, expert_bytes, order, offsets, pairs, top_k, n, k, flags, y, y_dtype),
      x_bf16, as_stream(stream)));
}

int moe_gemm_w4a4(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_tensor_scale,
                  const void* experts, int64_t n_experts, int64_t expert_bytes, const int32_t* order,
                  const int32_t* offsets, int64_t pairs, int64_t top_k, int64_t n, int64_t k,
                  unsigned flags, void* y, int y_dtype, void* stream) {
  const int st = check_product(pairs, top_k, n_experts, expert_bytes, QL_NVFP4, n, k, flags, y_dtype);
  if (st >= QL_OK) return st;
  // a row's place among the codes is a 31-bit offset
  const int64_t rows = flags & QL_ROWS_GATHER ? pairs / top_k : pairs;
  if (rows > (int64_t(1) << 32) / k - 1) return QL_ESHAPE;
  // a block of 512 threads for each tile, and room for one more to a CU
  if (w4a4_tiles(pairs, n_experts, n) > (int64_t(1) << 23) - 4096) return QL_ESHAPE;
  if (!a_codes || !a_scales || !a_tensor_scale || !experts || !offsets || !y ||
      (!order && (flags & QL_ROWS_GATHER)))
    return QL_EINVAL;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(experts) || !aligned16(y) ||
      !aligned(a_tensor_scale, 4) || !aligned(order, 4) || !aligned(offsets, 4))
    return QL_EALIGN;
  const Rows out = written(pairs, n, flags, y, y_dtype);
  if (overlap(out, whole(a_codes, rows, k / 2)) || overlap(out, whole(a_scales, rows, k / 16))) return QL_EINVAL;
  return launch_status(launch_moe_gemm_w4a4(
      product(experts, n_experts, expert_bytes, order, offsets, pairs, top_k, n, k, flags, y, y_dtype),
      a_codes, a_scales, a_tensor_scale, as_stream(stream)));
}

int moe_combine(const void* rows, int x_dtype, const int32_t* where, const int32_t* offsets,
                int64_t n_experts, const float* weights, int64_t tokens, int64_t top_k, int64_t n,
                void* out, int out_dtype, void* stream) {
  if (tokens < 0 || n < 0) return QL_EINVAL;
  if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return QL_EDTYPE;
  if (!groups_ok(n_experts) || top_k < 1 || top_k > kMostTopK || tokens > kMostRows / top_k) return QL_ESHAPE;
  if (n % 8 || n > (int64_t(1) << 24)) return QL_ESHAPE;
  if (tokens == 0 || n == 0) return QL_OK;
  if (!rows || !where || !offsets || !weights || !out) return QL_EINVAL;
  if (!aligned16(rows) || !aligned16(out) || !aligned(where, 4) || !aligned(offsets, 4) || !aligned(weights, 4))
    return QL_EALIGN;
  if (overlap(whole(out, tokens, n * bytes_of(out_dtype)), whole(rows, tokens * top_k, n * bytes_of(x_dtype))))
    return QL_EINVAL;
  const RowPlan p{nullptr, offsets, int(n_experts), int(tokens * top_k)};
  return launch_status(launch_moe_combine(rows, x_dtype, p, where, weights, tokens, int(top_k), n, out,
                                          out_dtype, as_stream(stream)));
}

size_t lora_add_workspace(int64_t rows, int64_t adapters, int64_t rank, int64_t k) {
  if (rows <= 0 || rows > kMostRows || !groups_ok(adapters) || rank < 8 || rank > 128 || rank % 8 ||
      k < 128 || k % 128 || k > (int64_t(1) << 20))
    return 0;
  return lora_ws_bytes(rows, adapters, int(rank), k);
}

int lora_add(const void* y, int64_t y_stride, const void* x_bf16, int64_t x_stride, const void* a_bf16,
             const void* b_bf16, const float* scale, int64_t adapters, int64_t rank,
             const int32_t* order, const int32_t* offsets, int64_t rows, int64_t n, int64_t k, void* out,
             int64_t out_stride, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (rows < 0 || n < 0 || k < 0) return QL_EINVAL;
  if (!dtype_ok(y_dtype)) return QL_EDTYPE;
  if (!groups_ok(adapters) || rank < 8 || rank > 128 || rank % 8 || rows > kMostRows) return QL_ESHAPE;
  if (n == 0 || k == 0 || n % 16 || k % 128 || n > (int64_t(1) << 24) || k > (int64_t(1) << 20)) return QL_ESHAPE;
  const int64_t size = bytes_of(y_dtype);
  const int64_t most = kMostSpan / (rows ? rows : 1);   // bytes between rows
  if (x_stride < k || y_stride < n || out_stride < n || x_stride > most / 2 || y_stride > most / size ||
      out_stride > most / size)
    return QL_ESHAPE;
  if (x_stride * 2 % 16 || y_stride * size % 16 || out_stride * size % 16) return QL_EALIGN;
  if (rows == 0) return QL_OK;
  if (!y || !x_bf16 || !a_bf16 || !b_bf16 || !order || !offsets || !out) return QL_EINVAL;
  if (!aligned16(y) || !aligned16(x_bf16) || !aligned16(a_bf16) || !aligned16(b_bf16) || !aligned16(out) ||
      !aligned(scale, 4) || !aligned(order, 4) || !aligned(offsets, 4))
    return QL_EALIGN;
  if (out == y && out_stride != y_stride) return QL_EINVAL;
  const int st = check_workspace(lora_add_workspace(rows, adapters, rank, k), workspace, workspace_bytes);
  if (st != QL_OK) return st;
  const Rows to{out, rows, out_stride * size, n * size};
  if (out != y && overlap(to, Rows{y, rows, y_stride * size, n * size})) return QL_EINVAL;
  if (overlap(to, Rows{x_bf16, rows, x_stride * 2, k * 2})) return QL_EINVAL;   // x of other blocks' rows
  LoraArgs g{};
  g.plan = RowPlan{order, offsets, int(adapters), int(rows)};
  g.x = x_bf16;
  g.a = a_bf16;
  g.b = b_bf16;
  g.y = y;
  g.scale = scale;
  g.out = out;
  g.x_stride = x_stride;
  g.y_stride = y_stride;
  g.out_stride = out_stride;
  g.rank = int(rank);
  g.n = int(n);
  g.k = int(k);
  g.y_dtype = y_dtype;
  g.part = static_cast<float*>(workspace);
  return launch_status(launch_lora_add(g, as_stream(stream)));
}

}  // extern "C"
