// extern "C" entry points of the paged key/value cache: argument validation
// and dispatch.  As in api.cpp every check runs on the host before any device
// work.  See include/qlin.h for the contract.
#include "kv_cache.hpp"

using namespace qlin;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int launch_status(hipError_t e) { return e == hipSuccess ? QL_OK : QL_EHIP; }

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t kMost = 0x7FFFFFFF;      // tokens, sequences, pages

bool sizes_ok(int64_t n_pages, int64_t page_size, int64_t n_kv, int64_t head_dim) {
  if (n_pages < 1 || n_pages > kMost || n_kv < 1 || n_kv > 1024) return false;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return false;
  if (page_size < 16 || page_size > 4096 || (page_size & (page_size - 1))) return false;
  return n_pages * n_kv <= (int64_t(1) << 40) / (page_size / 16);
}

bool format_ok(int f) { return f == QL_KV_BF16 || f == QL_KV_E4M3 || f == QL_KV_NVFP4; }

int64_t blocks_of(int64_t n_pages, int64_t page_size, int64_t n_kv) {
  return n_pages * n_kv * (page_size / 16);
}

// QL_OK and the geometry, or an error.
int check_cache(const ql_kv_cache* c, KvGeom* g) {
  if (!c) return QL_EINVAL;
  if (!format_ok(c->format)) return QL_EFORMAT;
  if (!sizes_ok(c->n_pages, c->page_size, c->n_kv, c->head_dim)) return QL_ESHAPE;
  if (!c->data) return QL_EINVAL;
  if (!aligned16(c->data)) return QL_EALIGN;
  if (c->bytes < kv_cache_bytes(c->format, c->n_pages, c->page_size, c->n_kv, c->head_dim))
    return QL_EWORKSPACE;
  g->codes = static_cast<uint8_t*>(c->data);
  g->scales = g->codes + blocks_of(c->n_pages, c->page_size, c->n_kv) * 32 *
                             kv_row_bytes(c->format, c->head_dim);
  g->n_pages = c->n_pages;
  g->n_kv = c->n_kv;
  g->page_shift = __builtin_ctz(unsigned(c->page_size));
  return QL_OK;
}

int esize(int dtype) { return dtype == QL_F32 ? 4 : 2; }

bool dtype_ok(int d) { return d == QL_F32 || d == QL_BF16; }

// Rows `stride` elements apart that hold `width` elements and start on 16 bytes.
int check_rows(int64_t stride, int64_t width, int dtype) {
  if (stride < width || stride > (int64_t(1) << 40)) return QL_ESHAPE;
  return stride * esize(dtype) % 16 ? QL_EALIGN : QL_OK;
}

}  // namespace

extern "C" {

size_t kv_cache_bytes(int format, int64_t n_pages, int64_t page_size, int64_t n_kv,
                      int64_t head_dim) {
  if (!format_ok(format) || !sizes_ok(n_pages, page_size, n_kv, head_dim)) return 0;
  return size_t(blocks_of(n_pages, page_size, n_kv)) *
         size_t(32 * kv_row_bytes(format, head_dim) + kv_scale_bytes(format, head_dim));
}

int kv_append(const ql_kv_cache* cache, const void* k, const void* v, int x_dtype,
              int64_t tokens, int64_t k_stride, int64_t v_stride, const int64_t* slots,
              void* stream) {
  KvGeom g;
  int st = check_cache(cache, &g);
  if (st != QL_OK) return st;
  if (tokens < 0) return QL_EINVAL;
  if (!dtype_ok(x_dtype)) return QL_EDTYPE;
  if (tokens > kMost) return QL_ESHAPE;
  const int64_t width = int64_t(cache->n_kv) * cache->head_dim;
  if ((st = check_rows(k_stride, width, x_dtype)) != QL_OK) return st;
  if ((st = check_rows(v_stride, width, x_dtype)) != QL_OK) return st;
  if (tokens == 0) return QL_OK;
  if (!k || !v || !slots) return QL_EINVAL;
  if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 7u)) return QL_EALIGN;
  return launch_status(launch_kv_append(g, cache->format, cache->head_dim, k, v, x_dtype, tokens,
                                        k_stride, v_stride, slots, as_stream(stream)));
}

int kv_gather(const ql_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
              int y_dtype, void* stream) {
  KvGeom g;
  const int st = check_cache(cache, &g);
  if (st != QL_OK) return st;
  if (tokens < 0) return QL_EINVAL;
  if (!dtype_ok(y_dtype)) return QL_EDTYPE;
  if (tokens > kMost) return QL_ESHAPE;
  if (tokens == 0) return QL_OK;
  if (!k || !v || !slots) return QL_EINVAL;
  if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 7u)) return QL_EALIGN;
  return launch_status(launch_kv_gather(g, cache->format, cache->head_dim, slots, tokens, k, v,
                                        y_dtype, as_stream(stream)));
}

int qkv_norm_rope_append(const ql_kv_cache* cache, const void* qkv, int x_dtype, int64_t tokens,
                         int64_t row_stride, int64_t n_q, const float* q_weight,
                         const float* k_weight, float eps, const int32_t* positions,
                         const float* rope, int64_t max_pos, int64_t rot, unsigned flags,
                         void* q_out, const int64_t* slots, void* stream) {
  KvGeom g;
  int st = check_cache(cache, &g);
  if (st != QL_OK) return st;
  if (tokens < 0 || (flags & ~QL_ROPE_INTERLEAVED)) return QL_EINVAL;
  if (!dtype_ok(x_dtype)) return QL_EDTYPE;
  if (tokens > kMost || n_q < 1 || n_q > 65536) return QL_ESHAPE;
  if (rot < 0 || rot > cache->head_dim || rot % 2) return QL_ESHAPE;
  if (rot && (max_pos < 1 || max_pos > kMost)) return QL_ESHAPE;
  if ((st = check_rows(row_stride, (n_q + 2 * int64_t(cache->n_kv)) * cache->head_dim, x_dtype)) !=
      QL_OK)
    return st;
  if (tokens == 0) return QL_OK;
  if (!qkv || !q_out || !slots || (rot && (!positions || !rope))) return QL_EINVAL;
  if (!aligned16(qkv) || !aligned16(q_out)) return QL_EALIGN;
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return QL_EALIGN;
  if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(rope) |
       reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 3u)
    return QL_EALIGN;
  return launch_status(launch_qkv_norm_rope_append(
      g, cache->format, cache->head_dim, qkv, x_dtype, tokens, row_stride, int(n_q), q_weight,
      k_weight, eps, positions, rope, max_pos, int(rot), (flags & QL_ROPE_INTERLEAVED) != 0, q_out,
      slots, as_stream(stream)));
}

// Sizes of an attention call; -1 if they may be planned, a status otherwise.
static int check_attention(const ql_kv_cache* cache, int64_t tokens, int64_t n_q, int64_t n_seqs,
                           int64_t max_q, int64_t max_kv) {
  if (tokens < 0 || n_seqs < 0 || max_q < 0 || max_kv < 0) return QL_EINVAL;
  if (n_q < 1 || n_q > 65536 || n_q % cache->n_kv) return QL_ESHAPE;
  if (tokens > kMost || n_seqs > 65535 || max_q > kMost || max_kv > kMost - 4096) return QL_ESHAPE;
  if (tokens == 0 || n_seqs == 0 || max_q == 0) return QL_OK;
  const int64_t m = max_q < tokens ? max_q : tokens;
  if (m * n_q > kMost - 4096) return QL_ESHAPE;   // rows are counted in 32 bits
  const KvAttnPlan p = kv_attention_plan(cache->format, cache->head_dim, int(n_q), cache->n_kv, n_seqs,
                                         m, max_kv);
  if (p.row_blocks > (kMost / 16) / (p.parts * cache->n_kv)) return QL_ESHAPE;
  return -1;
}

size_t kv_attention_workspace(const ql_kv_cache* cache, int64_t tokens, int64_t n_q,
                              int64_t n_seqs, int64_t max_q, int64_t max_kv) {
  if (!cache || !format_ok(cache->format) ||
      !sizes_ok(cache->n_pages, cache->page_size, cache->n_kv, cache->head_dim))
    return 0;
  if (check_attention(cache, tokens, n_q, n_seqs, max_q, max_kv) != -1) return 0;
  const int64_t m = max_q < tokens ? max_q : tokens;
  const KvAttnPlan p = kv_attention_plan(cache->format, cache->head_dim, int(n_q), cache->n_kv, n_seqs,
                                         m, max_kv);
  return kv_attention_ws_bytes(p, n_seqs, m, int(n_q), cache->head_dim);
}

int kv_attention(const ql_kv_cache* cache, const void* q_bf16, int64_t q_stride, int64_t tokens,
                 int64_t n_q, int64_t n_seqs, const int32_t* cu_q, const int32_t* kv_lens,
                 const int32_t* block_table, int64_t table_stride, int64_t table_cols,
                 int64_t max_q, int64_t max_kv, const uint64_t* tree, float scale, void* y,
                 void* workspace, size_t workspace_bytes, void* stream) {
  KvGeom g;
  int st = check_cache(cache, &g);
  if (st != QL_OK) return st;
  st = check_attention(cache, tokens, n_q, n_seqs, max_q, max_kv);
  if (st > QL_OK) return st;
  if (tree && max_q > 64) return QL_ESHAPE;
  if (table_cols < 0 || table_cols > kMost / cache->page_size || table_stride < table_cols ||
      table_stride > kMost)
    return QL_ESHAPE;
  const int rows = check_rows(q_stride, n_q * cache->head_dim, QL_BF16);
  if (rows != QL_OK) return rows;
  if (st == QL_OK) return QL_OK;
  if (!q_bf16 || !cu_q || !kv_lens || !y || (table_cols && !block_table)) return QL_EINVAL;
  if (!aligned16(q_bf16) || !aligned16(y) || (reinterpret_cast<uintptr_t>(tree) & 7u))
    return QL_EALIGN;
  if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(kv_lens) |
       reinterpret_cast<uintptr_t>(block_table)) & 3u)
    return QL_EALIGN;
  const int64_t m = max_q < tokens ? max_q : tokens;
  const KvAttnPlan p = kv_attention_plan(cache->format, cache->head_dim, int(n_q), cache->n_kv, n_seqs,
                                         m, max_kv);
  const size_t need = kv_attention_ws_bytes(p, n_seqs, m, int(n_q), cache->head_dim);
  if (need) {
    if (!workspace) return QL_EINVAL;
    if (!aligned16(workspace)) return QL_EALIGN;
    if (workspace_bytes < need) return QL_EWORKSPACE;
  }
  KvAttnArgs a{};
  a.g = g;
  a.q = q_bf16;
  a.q_stride = q_stride;
  a.tokens = tokens;
  a.n_seqs = int(n_seqs);
  a.n_q = int(n_q);
  a.cu_q = cu_q;
  a.kv_lens = kv_lens;
  a.table = block_table;
  a.table_stride = table_stride;
  a.table_cols = table_cols;
  a.max_q = int(m);
  a.max_kv = max_kv;
  a.tree = tree;
  a.scale = scale;
  a.y = y;
  a.part_o = static_cast<float*>(workspace);
  if (need) {
    a.part_ml = a.part_o + p.parts * m * n_q * cache->head_dim;
    a.first = reinterpret_cast<int32_t*>(a.part_ml + p.parts * m * n_q * 2);
  }
  a.parts = int(p.parts);
  return launch_status(launch_kv_attention(cache->format, cache->head_dim, p, a,
                                           as_stream(stream)));
}

int kv_commit(const ql_kv_cache* cache, int64_t n_seqs, const int32_t* cu_q,
              const int32_t* kv_lens, const int32_t* block_table, int64_t table_stride,
              int64_t table_cols, const int32_t* path, int64_t max_path, void* stream) {
  KvGeom g;
  const int st = check_cache(cache, &g);
  if (st != QL_OK) return st;
  if (n_seqs < 0 || max_path < 0) return QL_EINVAL;
  if (n_seqs > 65535 || max_path > 64) return QL_ESHAPE;
  if (table_cols < 0 || table_cols > kMost / cache->page_size || table_stride < table_cols ||
      table_stride > kMost)
    return QL_ESHAPE;
  if (n_seqs == 0 || max_path == 0) return QL_OK;
  if (!cu_q || !kv_lens || !path || (table_cols && !block_table)) return QL_EINVAL;
  if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(kv_lens) |
       reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(path)) & 3u)
    return QL_EALIGN;
  return launch_status(launch_kv_commit(g, cache->format, cache->head_dim, n_seqs, cu_q, kv_lens,
                                        block_table, table_stride, table_cols, path, int(max_path),
                                        as_stream(stream)));
}

}  // extern "C"
