// Drafted trees around the attention: rotation and append of a tree's rows,
// and the path that the model's own tokens confirm with the move of its keys
// and values.  Neither sums across rows.
#include <math.h>

#include <cmath>

#include "common.cuh"
#include "rope.cuh"
#include "tree.cuh"

namespace kinv {
namespace {

// A block per (node, heads of its row, sequence), a warp per head in turn.  A
// warp requests its first kRopeAhead heads before anything else is known of the
// tree than the node's row; meanwhile one warp finds the node's depth and then
// D/2 threads form the rotation's angles in fp64; the heads go through the code
// of kinv_rope_append.
constexpr int kRopeThreads = 256;
constexpr int kRopeAhead = 6;
constexpr int kRopeWholeRows = 128;  // from this many rows on a block takes a row whole (measured at the launch)

template <int D>
__global__ void __launch_bounds__(kRopeThreads)
    rope_append_tree_kernel(const __nv_bfloat16* __restrict__ qkv, int64_t ld_qkv,
                            __nv_bfloat16* __restrict__ q_out, __nv_bfloat16* __restrict__ k_cache,
                            __nv_bfloat16* __restrict__ v_cache, int64_t seq_stride, int64_t tok_stride,
                            const kinv_tree tree, const __nv_bfloat16* __restrict__ q_norm,
                            const __nv_bfloat16* __restrict__ k_norm, float eps, int Hq, int Hkv,
                            int heads_per_block, int* status, const RopeFreqs freqs) {
  constexpr int HALF = D / 2;
  constexpr int P = D / 64;  // pairs per lane
  constexpr int WARPS = kRopeThreads / 32;
  __shared__ TreeInfo ti;
  __shared__ float cs[HALF], sn[HALF];
  pdl_launch_dependents();
  pdl_wait();
  const int node = blockIdx.x, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n, ctx, off;
  if (!tree_bounds(tree, b, n, ctx, off)) {
    if (threadIdx.x == 0 && node == 0 && blockIdx.y == 0 && status) atomicExch(status, DEV_TREE_BAD);
    return;
  }
  if (node >= n) return;
  const int64_t r = off + node;
  const __nv_bfloat16* row = qkv + r * ld_qkv;
  const int64_t slot = b * seq_stride + static_cast<int64_t>(ctx + node) * tok_stride;
  const int heads = Hq + 2 * Hkv;
  const int h_end = min(heads, (static_cast<int>(blockIdx.y) + 1) * heads_per_block);
  // a lane's P values of each half of a head (for a value head likewise: D bits copied)
  uint32_t lo[kRopeAhead], hi[kRopeAhead];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) {
      const int h = h0 + i * WARPS;
      if (h >= h_end) continue;
      const __nv_bfloat16* src = row + h * D + lane * P;
      if (P == 2) {
        lo[i] = *reinterpret_cast<const uint32_t*>(src);
        hi[i] = *reinterpret_cast<const uint32_t*>(src + HALF);
      } else {
        lo[i] = *reinterpret_cast<const uint16_t*>(src);
        hi[i] = *reinterpret_cast<const uint16_t*>(src + HALF);
      }
    }
  };
  int h0 = blockIdx.y * heads_per_block + warp;
  load(h0);
  if (warp == 0) tree_load(tree, b, ti);
  __syncthreads();
  if (!ti.ok) {
    if (threadIdx.x == 0 && node == 0 && blockIdx.y == 0 && status) atomicExch(status, DEV_TREE_BAD);
    return;
  }
  const int p = ctx + __popcll(ti.mask[node]) - 1;
  if (threadIdx.x < HALF) rope_angle(p, freqs.inv_freq[threadIdx.x], cs[threadIdx.x], sn[threadIdx.x]);
  __syncthreads();
  float c[P], sv[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    c[j] = cs[lane * P + j];
    sv[j] = sn[lane * P + j];
  }
  for (; h0 < h_end; h0 += kRopeAhead * WARPS) {
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) {
      const int h = h0 + i * WARPS;
      if (h >= h_end) continue;
      if (h >= Hq + Hkv) {
        __nv_bfloat16* dst = v_cache + slot + (h - Hq - Hkv) * D + lane * P;
        if (P == 2) {
          *reinterpret_cast<uint32_t*>(dst) = lo[i];
          *reinterpret_cast<uint32_t*>(dst + HALF) = hi[i];
        } else {
          *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(lo[i]);
          *reinterpret_cast<uint16_t*>(dst + HALF) = static_cast<uint16_t>(hi[i]);
        }
        continue;
      }
      float a[P], bb[P];
      a[0] = bf16_lo(lo[i]);
      bb[0] = bf16_lo(hi[i]);
      if (P == 2) {
        a[P - 1] = bf16_hi(lo[i]);
        bb[P - 1] = bf16_hi(hi[i]);
      }
      __nv_bfloat16* dst = h < Hq ? q_out + (r * Hq + h) * D : k_cache + slot + (h - Hq) * D;
      rope_norm_rotate<D>(a, bb, c, sv, h < Hq ? q_norm : k_norm, eps, lane, dst);
    }
    load(h0 + kRopeAhead * WARPS);
  }
}

// A block per (layer and cache, sequence).  Every block finds the path itself:
// one warp, two nodes per lane, a ballot per step.  Then the path's slots are
// moved in ascending depth, a thread per 16-byte chunk of a slot; a source
// slot is never below its target (path[t] >= t), so no source is overwritten
// before it has been read.
constexpr int kAcceptThreads = 128;
constexpr int kAcceptAhead = 8;  // slots loaded before the first of them is stored

__global__ void __launch_bounds__(kAcceptThreads)
    tree_accept_kernel(const kinv_tree tree, const int32_t* __restrict__ tokens,
                       const int32_t* __restrict__ next_tokens, __nv_bfloat16* k_cache,
                       __nv_bfloat16* v_cache, int n_layers, int64_t layer_stride, int64_t seq_stride,
                       int64_t tok_stride, int chunks, int32_t* __restrict__ n_accepted,
                       int32_t* __restrict__ path_out, int32_t* __restrict__ out_tokens, int mark, int* status) {
  __shared__ int path[kTreeMaxNodes];
  __shared__ int s_len, s_ctx;
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int n, ctx, off;
    bool ok = tree_bounds(tree, b, n, ctx, off);
    int p[2] = {-2, -2}, tok[2] = {0, 0}, nxt[2] = {0, 0};
    if (ok) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        if (j < n) {
          p[i] = tree.parent[off + j];
          tok[i] = tokens[off + j];
          nxt[i] = next_tokens[off + j];
          ok = ok && p[i] >= -1 && p[i] < j;
        }
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    int len = ok ? 0 : -1;
    if (ok && n > 0) {
      int at = 0;
      while (true) {  // a child's index is above its parent's: at most n steps
        if (lane == 0) path[len] = at;
        ++len;
        const int want = __shfl_sync(0xffffffffu, at < 32 ? nxt[0] : nxt[1], at & 31);
        const unsigned lo = __ballot_sync(0xffffffffu, p[0] == at && tok[0] == want);
        const unsigned hi = __ballot_sync(0xffffffffu, p[1] == at && tok[1] == want);
        if (!(lo | hi)) break;
        at = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
      }
    }
    if (blockIdx.x == 0) {
      if (ok) {
        __syncwarp();
        if (lane == 0) n_accepted[b] = len;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = lane + 32 * i;
          const int j = t < len ? path[t] : 0;
          const int from_lo = __shfl_sync(0xffffffffu, nxt[0], j & 31);
          const int from_hi = __shfl_sync(0xffffffffu, nxt[1], j & 31);
          if (t < tree.max_nodes) {
            path_out[static_cast<int64_t>(b) * tree.max_nodes + t] = t < len ? j : -1;
            out_tokens[static_cast<int64_t>(b) * tree.max_nodes + t] = t < len ? (j < 32 ? from_lo : from_hi) : -1;
          }
        }
      } else {  // left out: marked where the caller asks for it
        if (lane == 0 && status) atomicExch(status, DEV_TREE_BAD);
        if (lane == 0 && (mark & KINV_TREE_MARK_COUNT)) n_accepted[b] = 0;
        for (int t = lane; t < tree.max_nodes; t += 32) {
          if (mark & KINV_TREE_MARK_PATH) path_out[static_cast<int64_t>(b) * tree.max_nodes + t] = -1;
          if (mark & KINV_TREE_MARK_TOKENS) out_tokens[static_cast<int64_t>(b) * tree.max_nodes + t] = -1;
        }
      }
    }
    if (lane == 0) {
      s_len = len;
      s_ctx = ctx;
    }
  }
  __syncthreads();
  const int len = s_len;
  const int layer = blockIdx.x >> 1;
  if (layer >= n_layers) return;
  __nv_bfloat16* base = (blockIdx.x & 1 ? v_cache : k_cache) + layer * layer_stride + b * seq_stride +
                        static_cast<int64_t>(s_ctx) * tok_stride;
  for (int c = threadIdx.x; c < chunks; c += kAcceptThreads) {
    for (int t0 = 1; t0 < len; t0 += kAcceptAhead) {
      uint4 v[kAcceptAhead];
#pragma unroll
      for (int i = 0; i < kAcceptAhead; ++i)
        if (t0 + i < len) v[i] = reinterpret_cast<const uint4*>(base + path[t0 + i] * tok_stride)[c];
#pragma unroll
      for (int i = 0; i < kAcceptAhead; ++i)
        if (t0 + i < len && path[t0 + i] != t0 + i) reinterpret_cast<uint4*>(base + (t0 + i) * tok_stride)[c] = v[i];
    }
  }
}

}  // namespace
}  // namespace kinv

using namespace kinv;

extern "C" kinv_status kinv_rope_append_tree(const void* qkv, int64_t ld_qkv, void* q_out, void* k_cache,
                                             void* v_cache, int64_t seq_stride, int64_t tok_stride,
                                             const kinv_tree* tree, const void* q_norm, const void* k_norm,
                                             float eps, int Hq, int Hkv, int D, float rope_base,
                                             kinv_stream stream) {
  const kinv_status st = tree_check(tree);
  if (st != KINV_OK) return st;
  if (Hq <= 0 || Hkv <= 0 || !(rope_base > 0.f) || !(eps >= 0.f)) return KINV_ERR_INVALID_ARG;
  if (tree_empty(tree)) return KINV_OK;
  if (!qkv || !q_out || !k_cache || !v_cache) return KINV_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return KINV_ERR_UNSUPPORTED;
  if (ld_qkv < static_cast<int64_t>(Hq + 2 * Hkv) * D || tok_stride < static_cast<int64_t>(Hkv) * D ||
      seq_stride < 0 || (tree->B > 1 && seq_stride == 0))
    return KINV_ERR_INVALID_ARG;
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) || ld_qkv % 8 ||
      seq_stride % 8 || tok_stride % 8)
    return KINV_ERR_ALIGNMENT;
  // the frequencies of the last base and head size this thread used
  static thread_local struct {
    float base;
    int D;
    RopeFreqs f;
  } last = {0.f, 0, {}};
  if (last.base != rope_base || last.D != D) {
    for (int i = 0; i < D / 2; ++i) last.f.inv_freq[i] = std::pow(static_cast<double>(rope_base), -2.0 * i / D);
    last.base = rope_base;
    last.D = D;
  }
  const RopeFreqs& freqs = last.f;
  const int heads = Hq + 2 * Hkv;
  // A head per warp while the rows leave SMs free, whole rows behind that, where the
  // angles, formed once per block, and the blocks themselves count (48 heads of 128,
  // rows: us with 8 heads a block / with all: 8: 3.7 / 5.0, 64: 4.7 / 5.5, 128: 5.6 /
  // 5.6, 256: 8.3 / 5.9, 512: 13.4 / 8.4, 2,048: 43 / 17.7; 16 and 24 heads a block lie
  // between the two from 256 rows).
  const int hpb = tree->total_rows >= kRopeWholeRows ? heads : 8;
  const dim3 grid(tree->max_nodes, (heads + hpb - 1) / hpb, tree->B);
  int* status = device_status_word();
  auto* k = static_cast<__nv_bfloat16*>(k_cache);
  auto* v = static_cast<__nv_bfloat16*>(v_cache);
  auto* src = static_cast<const __nv_bfloat16*>(qkv);
  auto* qo = static_cast<__nv_bfloat16*>(q_out);
  auto* qn = static_cast<const __nv_bfloat16*>(q_norm);
  auto* kn = static_cast<const __nv_bfloat16*>(k_norm);
  auto* kernel = D == 128 ? rope_append_tree_kernel<128> : rope_append_tree_kernel<64>;
  return launch_kernel(kernel, grid, dim3(kRopeThreads), 0, stream, 1, src, ld_qkv, qo, k, v, seq_stride, tok_stride,
                       *tree, qn, kn, eps, Hq, Hkv, hpb, status, freqs);
}

extern "C" kinv_status kinv_tree_accept(const kinv_tree* tree, const int32_t* tokens,
                                        const int32_t* next_tokens, void* k_cache, void* v_cache,
                                        int n_layers, int64_t layer_stride, int64_t seq_stride,
                                        int64_t tok_stride, int Hkv, int D, int32_t* n_accepted,
                                        int32_t* path, int32_t* out_tokens, kinv_stream stream) {
  return kinv_tree_accept_marked(tree, tokens, next_tokens, k_cache, v_cache, n_layers, layer_stride, seq_stride,
                                 tok_stride, Hkv, D, n_accepted, path, out_tokens, 0, stream);
}

extern "C" kinv_status kinv_tree_accept_marked(const kinv_tree* tree, const int32_t* tokens,
                                               const int32_t* next_tokens, void* k_cache, void* v_cache,
                                               int n_layers, int64_t layer_stride, int64_t seq_stride,
                                               int64_t tok_stride, int Hkv, int D, int32_t* n_accepted,
                                               int32_t* path, int32_t* out_tokens, int mark,
                                               kinv_stream stream) {
  const kinv_status st = tree_check(tree);
  if (st != KINV_OK) return st;
  if (n_layers < 0 || (mark & ~(KINV_TREE_MARK_COUNT | KINV_TREE_MARK_PATH | KINV_TREE_MARK_TOKENS)))
    return KINV_ERR_INVALID_ARG;
  if (n_layers > 65535) return KINV_ERR_UNSUPPORTED;
  if (tree->B == 0) return KINV_OK;
  if (!n_accepted) return KINV_ERR_INVALID_ARG;
  if (tree->max_nodes > 0 && (!path || !out_tokens)) return KINV_ERR_INVALID_ARG;
  if (tree_empty(tree)) {  // no sequence may have a node: the arrays of the tree are not needed
    if (tree->max_nodes > 0 &&
        (cudaMemsetAsync(path, 0xFF, sizeof(int32_t) * tree->B * tree->max_nodes, stream) != cudaSuccess ||
         cudaMemsetAsync(out_tokens, 0xFF, sizeof(int32_t) * tree->B * tree->max_nodes, stream) != cudaSuccess))
      return KINV_ERR_CUDA;
    return cuda_status(cudaMemsetAsync(n_accepted, 0, sizeof(int32_t) * tree->B, stream));
  }
  if (!tokens || !next_tokens) return KINV_ERR_INVALID_ARG;
  int chunks = 0;
  if (n_layers > 0) {
    if (!k_cache || !v_cache || Hkv <= 0 || D <= 0) return KINV_ERR_INVALID_ARG;
    if (D % 8) return KINV_ERR_UNSUPPORTED;
    if (tok_stride < static_cast<int64_t>(Hkv) * D || seq_stride < 0 || layer_stride < 0 ||
        (tree->B > 1 && seq_stride == 0) || (n_layers > 1 && layer_stride == 0))
      return KINV_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || layer_stride % 8 || seq_stride % 8 || tok_stride % 8)
      return KINV_ERR_ALIGNMENT;
    chunks = static_cast<int>(static_cast<int64_t>(Hkv) * D / 8);
  }
  const dim3 grid(n_layers > 0 ? 2 * n_layers : 1, tree->B);
  return launch_kernel(tree_accept_kernel, grid, dim3(kAcceptThreads), 0, stream, 1, *tree, tokens, next_tokens,
                       static_cast<__nv_bfloat16*>(k_cache), static_cast<__nv_bfloat16*>(v_cache), n_layers,
                       layer_stride, seq_stride, tok_stride, chunks, n_accepted, path, out_tokens, mark,
                       device_status_word());
}
