// A batch of trees of drafted tokens (kinv_tree) as the kernels read it.
#pragma once

#include "common.cuh"

namespace kinv {

constexpr int kTreeMaxNodes = KINV_TREE_MAX_NODES;
static_assert(kTreeMaxNodes == 64, "a node's ancestors are a 64-bit mask, two nodes per lane of a warp");

constexpr int DEV_TREE_BAD = dev_code(8, KINV_ERR_INVALID_ARG);

// A sequence's tree in shared memory.
struct TreeInfo {
  unsigned long long mask[kTreeMaxNodes];  // bit j of node i: j is i or an ancestor of i
  int n, ctx, off;                         // nodes, keys before the tree, row of node 0
  int ok;                                  // the sequence keeps its stated bounds
};

// Sequence b's device-side numbers within the stated bounds?  (No parent is read.)
__device__ __forceinline__ bool tree_bounds(const kinv_tree& t, int b, int& n, int& ctx, int& off) {
  n = t.n_nodes[b];
  ctx = t.ctx_len[b];
  off = t.row_offset[b];
  return n >= 0 && n <= t.max_nodes && ctx >= 0 && ctx <= t.max_kv - n && off >= 0 && off <= t.total_rows - n;
}

// Loads sequence b's tree; called by all 32 lanes of one warp, the results
// visible to the block after its next barrier.  Lane l holds nodes l and
// l + 32.  Each node's ancestors by pointer doubling: after round r a node
// knows its nearest 2^r ancestors and points at the next one, so ceil(log2 n)
// rounds reach the root whatever the tree's shape.  A parent has the lower
// index, so ascending bits of a mask are ascending depths and the t-th set bit
// is the path's node at depth t.
__device__ __forceinline__ void tree_load(const kinv_tree& t, int b, TreeInfo& s) {
  const int lane = threadIdx.x & 31;
  int n, ctx, off;
  bool ok = tree_bounds(t, b, n, ctx, off);
  int p0 = -1, p1 = -1;
  if (ok && lane < n) {
    p0 = t.parent[off + lane];
    ok = p0 >= -1 && p0 < lane;
  }
  if (ok && lane + 32 < n) {
    p1 = t.parent[off + lane + 32];
    ok = p1 >= -1 && p1 < lane + 32;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) p0 = p1 = -1;
  unsigned long long m0 = 1ull << lane, m1 = 1ull << (lane + 32);
  const int top = ok ? n : 0;
  for (int span = 1; span < top; span <<= 1) {
    // p0 < lane < 32: the low half's parents lie in the low half
    const unsigned long long a0 = __shfl_sync(0xffffffffu, m0, p0 & 31);
    const int q0 = __shfl_sync(0xffffffffu, p0, p0 & 31);
    const unsigned long long a1 = __shfl_sync(0xffffffffu, m0, p1 & 31), b1 = __shfl_sync(0xffffffffu, m1, p1 & 31);
    const int q1 = __shfl_sync(0xffffffffu, p0, p1 & 31), r1 = __shfl_sync(0xffffffffu, p1, p1 & 31);
    if (p1 >= 0) {
      m1 |= p1 < 32 ? a1 : b1;
      p1 = p1 < 32 ? q1 : r1;
    }
    if (p0 >= 0) {
      m0 |= a0;
      p0 = q0;
    }
  }
  s.mask[lane] = m0;
  s.mask[lane + 32] = m1;
  if (lane == 0) {
    s.n = n;
    s.ctx = ctx;
    s.off = off;
    s.ok = ok;
  }
}

// Host-side checks of a kinv_tree (no CUDA call is made).  KINV_OK with
// t.B, t.total_rows or t.max_nodes 0 means there is nothing to do.
inline kinv_status tree_check(const kinv_tree* t) {
  if (!t || t->B < 0 || t->total_rows < 0 || t->max_nodes < 0 || t->max_kv < 0) return KINV_ERR_INVALID_ARG;
  if (t->max_nodes > kTreeMaxNodes || t->B > 65535) return KINV_ERR_UNSUPPORTED;
  if (t->B == 0 || t->total_rows == 0 || t->max_nodes == 0) return KINV_OK;
  if (!t->ctx_len || !t->n_nodes || !t->row_offset || !t->parent) return KINV_ERR_INVALID_ARG;
  return KINV_OK;
}
inline bool tree_empty(const kinv_tree* t) { return t->B == 0 || t->total_rows == 0 || t->max_nodes == 0; }

}  // namespace kinv
