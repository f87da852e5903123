// Host-side checks that the calls around a round and those of a decoding step share.
#pragma once

#include <math.h>
#include <stdint.h>

#include "rounds.h"

namespace wf {

constexpr size_t kWorkspaceAlign = 256;
constexpr int64_t kMaxBlocks = int64_t{1} << 22;  // x 1024 threads: below 2^32 work items

constexpr int32_t kMaxVocab = 1 << 30;
constexpr int64_t kMaxPositions = 1 << 30;  // of a sequence: sums of two stay in an int

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
inline bool valid_dtype(int32_t d) { return d == WF_F32 || d == WF_BF16; }
inline int32_t elem_bytes(int32_t d) { return d == WF_BF16 ? 2 : 4; }
inline int32_t launch_status(hipError_t e) { return e == hipSuccess ? WF_OK : WF_ERR_LAUNCH; }

inline int32_t check_workspace(void* ws, size_t have, size_t need) {
  if (need == 0) return WF_OK;
  if (ws == nullptr || reinterpret_cast<uintptr_t>(ws) % kWorkspaceAlign != 0 || have < need)
    return WF_ERR_WORKSPACE;
  return WF_OK;
}

// Sizes of a round; *total gets its packed rows.
inline int32_t check_sizes(const wf_round_rows* r, int64_t* total) {
  if (!r) return WF_ERR_NULL;
  if (r->kind < WF_ROWS_CHAIN || r->kind > WF_ROWS_ROUTED || r->B < 0) return WF_ERR_SHAPE;
  const bool chain = r->kind != WF_ROWS_TREE, tree = r->kind != WF_ROWS_CHAIN;
  if (chain && (r->K < 0 || r->K >= WHIFLASH_MAX_SEQ_ROWS)) return WF_ERR_SHAPE;
  if (tree && (r->N < 1 || r->N > WHIFLASH_MAX_SEQ_ROWS)) return WF_ERR_SHAPE;
  if (r->kind == WF_ROWS_ROUTED && r->total_rows < 0) return WF_ERR_SHAPE;
  *total = r->kind == WF_ROWS_CHAIN  ? static_cast<int64_t>(r->B) * (r->K + 1)
           : r->kind == WF_ROWS_TREE ? static_cast<int64_t>(r->B) * r->N
                                     : r->total_rows;
  return *total > INT32_MAX ? WF_ERR_SHAPE : WF_OK;
}

inline RowsArgs rows_args(const wf_round_rows* r, int64_t total) {
  RowsArgs a{};
  a.kind = r->kind;
  a.B = r->B;
  a.K = r->kind != WF_ROWS_TREE ? r->K : 0;
  a.N = r->kind != WF_ROWS_CHAIN ? r->N : 0;
  a.Vd = r->Vd;
  a.total_rows = static_cast<int32_t>(total);
  const int32_t chain = r->kind != WF_ROWS_TREE ? a.K + 1 : 0;
  a.rmax = chain > a.N ? chain : a.N;
  a.chain_draft = r->chain_draft;
  a.parent = r->parent;
  a.draft_ids = r->draft_ids;
  a.d2t = r->d2t;
  a.row_offsets = r->row_offsets;
  a.choice = r->choice;
  return a;
}

// The round's pointers, after its sizes; `tokens`: the call reads draft tokens.
inline int32_t check_pointers(const wf_round_rows* r, bool tokens) {
  const bool chain = r->kind != WF_ROWS_TREE, tree = r->kind != WF_ROWS_CHAIN;
  if (r->kind == WF_ROWS_ROUTED && (!r->row_offsets || !r->choice)) return WF_ERR_NULL;
  if (tree && !r->parent) return WF_ERR_NULL;
  if (tokens && chain && r->K > 0 && !r->chain_draft) return WF_ERR_NULL;
  if (tokens && tree) {
    if (r->Vd < 1) return WF_ERR_SHAPE;
    if (!r->draft_ids || !r->d2t) return WF_ERR_NULL;
  }
  return WF_OK;
}

inline int32_t check_matrix(const void* p, int32_t dtype, int64_t rows, int32_t V, int64_t stride) {
  if (!valid_dtype(dtype)) return WF_ERR_DTYPE;
  if (V <= 0 || V > kMaxVocab || stride < V || stride > INT64_MAX / 16 / (rows > 0 ? rows : 1))
    return WF_ERR_SHAPE;
  if (rows > 0 && !p) return WF_ERR_NULL;
  if (!aligned16(p) || (stride * elem_bytes(dtype)) % 16 != 0) return WF_ERR_ALIGN;
  return WF_OK;
}

// A cache's sizes and pointers, its element type apart.
inline int32_t check_pages(const wf_page_cache* c, int32_t b) {
  if (c->layers < 1 || c->pages < 1 || c->heads < 1 || c->heads > 1024 || c->seqs < 1 ||
      c->max_pages < 1 || c->layers > 4096 || (c->head_dim != 64 && c->head_dim != 128) ||
      c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0 ||
      static_cast<int64_t>(c->max_pages) * c->page_size > kMaxPositions)
    return WF_ERR_SHAPE;
  const int64_t page = static_cast<int64_t>(c->heads) * c->page_size * c->head_dim;
  if (c->page_stride < page || c->page_stride > INT64_MAX / 16 / c->pages ||
      (c->layers > 1 && (c->layer_stride < page || c->layer_stride > INT64_MAX / 16 / c->layers)))
    return WF_ERR_SHAPE;
  if (!c->k || !c->v || !c->table || !c->held || !c->context || !c->refs) return WF_ERR_NULL;
  if (!aligned16(c->k) || !aligned16(c->v) || c->page_stride * b % 16 != 0 ||
      (c->layers > 1 && c->layer_stride * b % 16 != 0))
    return WF_ERR_ALIGN;
  return WF_OK;
}

inline int32_t check_cache(const wf_page_cache* c) {
  if (!c) return WF_ERR_NULL;
  if (!valid_dtype(c->dtype)) return WF_ERR_DTYPE;
  return check_pages(c, elem_bytes(c->dtype));
}

// ... for the calls that read no keys and values: the pages of an 8-bit cache too.
inline int32_t check_bookkeeping(const wf_page_cache* c) {
  return c && c->dtype == WF_E4M3 ? check_pages(c, 1) : check_cache(c);
}

// Rows of `width` elements (queries, new keys and values).
inline int32_t check_vectors(const void* p, int32_t dtype, int64_t rows, int64_t width, int64_t stride) {
  if (stride < width || stride > INT64_MAX / 16 / (rows > 0 ? rows : 1)) return WF_ERR_SHAPE;
  if (rows > 0 && !p) return WF_ERR_NULL;
  if (!aligned16(p) || stride * elem_bytes(dtype) % 16 != 0) return WF_ERR_ALIGN;
  return WF_OK;
}

// A cache call's round; *out is set for B > 0.
inline int32_t check_cache_rows(const wf_page_cache* cache, const wf_round_rows* rows, int64_t* total,
                         RowsArgs* out) {
  int32_t s = check_cache(cache);
  if (s != WF_OK) return s;
  if ((s = check_sizes(rows, total)) != WF_OK) return s;
  if (rows->B == 0) return WF_OK;
  if ((s = check_pointers(rows, false)) != WF_OK) return s;
  *out = rows_args(rows, *total);
  if (static_cast<int64_t>(rows->B) * out->rmax > kMaxBlocks) return WF_ERR_SHAPE;
  return WF_OK;
}

inline bool attend_sizes_ok(const wf_page_cache* c, int32_t q_heads, int32_t max_context) {
  return q_heads >= 1 && q_heads <= 65535 && q_heads % c->heads == 0 && max_context >= 0 &&
         max_context <= kMaxPositions;
}

}  // namespace wf
