// The rows of a round (wf_round_rows) as the kernels see them.
#pragma once

#include "common.h"

namespace wf {

struct RowsArgs {
  int kind, B, K, N, Vd, total_rows;
  int rmax;  // rows of the longest well-formed sequence
  const int32_t* chain_draft;
  const int32_t* parent;
  const int32_t* draft_ids;
  const int32_t* d2t;
  const int32_t* row_offsets;
  const int32_t* choice;
};

// One sequence's rows: [row0, row0 + n), as a tree or a chain; n = 0 if malformed.
struct SeqRows {
  int row0, n;
  bool tree;
};

__device__ inline SeqRows seq_rows(const RowsArgs& a, int b) {
  if (a.kind == WF_ROWS_CHAIN) return SeqRows{b * (a.K + 1), a.K + 1, false};
  if (a.kind == WF_ROWS_TREE) return SeqRows{b * a.N, a.N, true};
  const int lo = a.row_offsets[b], hi = a.row_offsets[b + 1], c = a.choice[b];
  const bool in_range = lo >= 0 && lo <= hi && hi <= a.total_rows;
  const int n = in_range ? hi - lo : 0;
  const bool ok = (c == 0 && n == a.K + 1) || (c == 1 && n == a.N);
  return SeqRows{lo, ok ? n : 0, c == 1};
}

// The parent of node u >= 1 of sequence b, or -1 where its path ends.
__device__ inline int node_parent(const RowsArgs& a, int b, bool tree, int u) {
  if (!tree) return u - 1;
  const int p = a.parent[static_cast<int64_t>(b) * a.N + u];
  return p >= 0 && p < u ? p : -1;
}

// The token that node u >= 1 of sequence b drafted, or -1 for none.
__device__ inline int node_token(const RowsArgs& a, int b, bool tree, int u, int V) {
  int t;
  if (tree) {
    const int id = a.draft_ids[static_cast<int64_t>(b) * a.N + u];
    t = id >= 0 && id < a.Vd ? a.d2t[id] : -1;
  } else {
    t = a.chain_draft[static_cast<int64_t>(b) * a.K + u - 1];
  }
  return t >= 0 && t < V ? t : -1;
}

// The slot of sequence b among `n` (map NULL: b itself), or -1.
__device__ inline int slot_of(const int32_t* map, int b, int n) {
  const int s = map ? map[b] : b;
  return s >= 0 && s < n ? s : -1;
}

}  // namespace wf
