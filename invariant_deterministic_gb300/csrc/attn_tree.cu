// Attention of drafted trees over a cache (kinv_attn_tree), with the decode
// kernel's arithmetic for every row: a node of depth t behind L context keys
// is the decode row of length L + t + 1 whose last t + 1 keys are its path.
//
// The keys are cut into splits of 256 at absolute positions.  Every node of a
// sequence sees the same keys in the splits that end within the context, so
// those take (row, query head) pairs of many nodes as the rows of one MMA.  In
// the one or two splits that hold path positions the scores of a pair against
// all drafted keys are formed once (a score depends only on its q and k rows)
// and each is put at its position; the 16-key steps of P.V that lie within the
// context stay shared, and a step that holds path positions runs once per node
// with that node's own V rows gathered through the addresses of ldmatrix,
// keeping only the node's accumulator rows.  So a pair's maximum, weights, sum
// order and P.V chain are those of the decode row.
#include <math.h>

#include "attn_mma.cuh"
#include "common.cuh"
#include "tree.cuh"

namespace kinv {
namespace {

constexpr int kSplit = 256;    // keys per split, as in decode and prefill
constexpr int kThreads = 256;  // eight warps, 32 positions each for the softmax
constexpr int kMaxG = 8;

struct TreeAttnParams {
  kinv_tree tree;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t seq_stride, tok_stride;
  __nv_bfloat16* out;
  float* ws_o;   // [total_rows][Hq][S][D]
  float* ws_ml;  // [total_rows][Hq][S][2]
  int Hq, Hkv, G;
  int S;         // splits per row in the workspace
  float c2;      // fp32(scale * log2 e) > 0
  int* status;
};

__device__ __forceinline__ void report_bad_tree(const TreeAttnParams& p) {
  if (threadIdx.x == 0 && p.status) atomicExch(p.status, DEV_TREE_BAD);
}

// One block per (kv head, tile of 16 MT pairs, split, sequence).
template <int D, int MT>
__global__ void __launch_bounds__(kThreads) attn_tree_split_kernel(const TreeAttnParams p) {
  constexpr int C8 = D / 8;   // 16-byte chunks per key row
  constexpr int KS = D / 16;  // 16-wide k steps of q . k
  constexpr int R = 16 * MT;  // pairs of the tile
  // rows of 16-byte chunks, chunk c of row r at chunk c ^ (r & 7): K, then V
  // (up to 256 context keys, or up to 255 and the drafted ones); the scores by
  // position [R][256] fp32, then P_hi and P_lo [R][256] in their place; the
  // path of each node of the tile; a row of zeros
  extern __shared__ __align__(16) unsigned char smem_raw[];
  constexpr int KV_ROWS = kSplit + kTreeMaxNodes;
  unsigned char* kv = smem_raw;
  unsigned char* pt = kv + KV_ROWS * D * 2;
  unsigned char* pt_lo = pt + R * kSplit * 2;
  float* scores = reinterpret_cast<float*>(pt);
  unsigned char* zrow = pt_lo + R * kSplit * 2;
  unsigned char* paths = zrow + D * 2;  // [R][64]
  __shared__ TreeInfo ti;
  __shared__ float wmax[kThreads / 32][R];
  __shared__ float wsum[kThreads / 32][R];

  pdl_launch_dependents();
  pdl_wait();
  const int g = blockIdx.x % p.Hkv;
  const int tile = blockIdx.x / p.Hkv;
  const int s = blockIdx.y;
  const int b = blockIdx.z;
  int n, ctx, off;
  if (!tree_bounds(p.tree, b, n, ctx, off)) {
    report_bad_tree(p);
    return;
  }
  const int G = p.G;
  const int npt = R / G;  // nodes of a tile
  const int n0 = tile * npt;
  const int k0 = s * kSplit;
  if (n0 >= n || k0 >= ctx + n) return;
  const int nodes = min(npt, n - n0);
  const int c = max(0, min(kSplit, ctx - k0));  // context keys of this split
  const bool tail = c < kSplit;
  const int t = threadIdx.x;
  const int lane = t & 31, warp = t >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int shift = k0 - ctx + c;  // path index of position k0 + c (0, or 256 - L % 256 in a second tail split)
  const uint32_t kv_base = smem_addr(kv), pt_base = smem_addr(pt), pt_lo_base = smem_addr(pt_lo);
  const uint32_t zrow_base = smem_addr(zrow);

  const int drafted = tail ? n0 + nodes : 0;  // ancestors have lower indices: later nodes are nobody's here
  const int rows = c + drafted;
  const int64_t seq_off = b * p.seq_stride + g * D;
  const uint64_t kv_policy = l2_policy_evict_first();
  auto load = [&](const __nv_bfloat16* src) {
    for (int idx = t; idx < rows * C8; idx += kThreads) {
      const int r = idx / C8, ch = idx % C8;
      const int slot = r < c ? k0 + r : ctx + r - c;
      cp_async16_hint(kv_base + static_cast<uint32_t>(r * D * 2 + ((ch ^ (r & 7)) << 4)),
                      src + seq_off + static_cast<int64_t>(slot) * p.tok_stride + ch * 8, kv_policy);
    }
    cp_async_commit();
  };
  load(p.k);

  if (tail) {
    if (warp == 0) tree_load(p.tree, b, ti);
    for (int i = t; i < D * 2 / 16; i += kThreads) *reinterpret_cast<uint4*>(zrow + 16 * i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (!ti.ok) {
      report_bad_tree(p);
      cp_async_wait<0>();
      return;
    }
    // the path of a node: the set bits of its mask, ascending
    for (int idx = t; idx < nodes * kTreeMaxNodes; idx += kThreads) {
      const int i = idx / kTreeMaxNodes, j = idx % kTreeMaxNodes;
      const unsigned long long m = ti.mask[n0 + i];
      if (m >> j & 1) paths[i * kTreeMaxNodes + __popcll(m & ((1ull << j) - 1))] = static_cast<unsigned char>(j);
    }
  }

  // q fragments (A operand), straight from global: MMA row r of tile mt is pair
  // 16 mt + r, node n0 + pair / G, query head g G + pair % G
  uint32_t qa[MT][KS][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r_lo = mt * 16 + gq, r_hi = r_lo + 8;
    auto row = [&](int r) -> const __nv_bfloat16* {
      return r / G < nodes ? p.q + (static_cast<int64_t>(off + n0 + r / G) * p.Hq + g * G + r % G) * D : nullptr;
    };
    const __nv_bfloat16 *q_lo = row(r_lo), *q_hi = row(r_hi);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int d0 = ks * 16 + 2 * tq;
      qa[mt][ks][0] = q_lo ? *reinterpret_cast<const uint32_t*>(q_lo + d0) : 0u;
      qa[mt][ks][1] = q_hi ? *reinterpret_cast<const uint32_t*>(q_hi + d0) : 0u;
      qa[mt][ks][2] = q_lo ? *reinterpret_cast<const uint32_t*>(q_lo + d0 + 8) : 0u;
      qa[mt][ks][3] = q_hi ? *reinterpret_cast<const uint32_t*>(q_hi + d0 + 8) : 0u;
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // scores of eight key rows (from `key0`) against the tile's pairs
  auto score_block = [&](int key0, float (&sc)[MT][4]) {
    const int key = key0 + (lane & 7);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[mt][i] = 0.f;
#pragma unroll
    for (int kp = 0; kp < KS / 2; ++kp) {
      const int ch = kp * 4 + (lane >> 3);
      uint32_t b0, b1, b2, b3;
      ldsm_x4(kv_base + static_cast<uint32_t>(key * D * 2 + ((ch ^ (key & 7)) << 4)), b0, b1, b2, b3);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma_bf16_16816(sc[mt], qa[mt][2 * kp], b0, b1);
        mma_bf16_16816(sc[mt], qa[mt][2 * kp + 1], b2, b3);
      }
    }
  };
  float sc[4][MT][4];  // warp w: positions 32w + 8nb + 2tq (+1), pairs gq and gq + 8 of each MMA tile
  int cnt[MT][2];      // positions of this split that the pair sees
  int cnt_max = 0;
  if (!tail) {
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) score_block(warp * 32 + nb * 8, sc[nb]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) cnt[mt][h] = (mt * 16 + h * 8 + gq) / G < nodes ? kSplit : 0;
    cnt_max = kSplit;
  } else {
    // every key row's scores, put at the position the key has for the pair
    for (int blk = warp; blk * 8 < rows; blk += kThreads / 32) {
      float one[MT][4];
      score_block(blk * 8, one);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pair = mt * 16 + gq + (i >> 1) * 8;
          const int key = blk * 8 + 2 * tq + (i & 1);
          if (pair / G >= nodes || key >= rows) continue;
          int at = key;
          if (key >= c) {
            const int j = key - c;
            if (!(ti.mask[n0 + pair / G] >> j & 1)) continue;
            at = c + __popcll(ti.mask[j]) - 1 - shift;
            if (at < c || at >= kSplit) continue;
          }
          scores[pair * kSplit + at] = one[mt][i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int pair = mt * 16 + h * 8 + gq;
        const int i = pair / G;
        cnt[mt][h] = i < nodes ? max(0, min(kSplit, ctx + __popcll(ti.mask[n0 + i]) - k0)) : 0;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = warp * 32 + nb * 8 + 2 * tq + e;
            sc[nb][mt][2 * h + e] = at < cnt[mt][h] ? scores[pair * kSplit + at] : 0.f;
          }
      }
    for (int i = 0; i < nodes; ++i) cnt_max = max(cnt_max, min(kSplit, ctx + __popcll(ti.mask[n0 + i]) - k0));
  }
  __syncthreads();  // every warp is done with K and with the scores' array
  load(p.v);

  // the decode kernel's statistics: raw maxima (exact in any order), m =
  // fp32(max * c), the weights, a lane's eight in (nb, e) order, the four
  // lanes, the eight warps
  float m[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = -INFINITY;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (warp * 32 + nb * 8 + 2 * tq + e < cnt[mt][h]) mx = fmaxf(mx, sc[nb][mt][2 * h + e]);
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (tq == 0) wmax[warp][mt * 16 + h * 8 + gq] = mx;
    }
  __syncthreads();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pair = mt * 16 + h * 8 + gq;
      float mm = wmax[0][pair];
#pragma unroll
      for (int w = 1; w < kThreads / 32; ++w) mm = fmaxf(mm, wmax[w][pair]);
      m[mt][h] = mm = __fmul_rn(mm, p.c2);
      float sum = 0.f;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        float x[2], hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[e] = warp * 32 + nb * 8 + 2 * tq + e < cnt[mt][h]
                     ? ex2_approx(__fmaf_rn(sc[nb][mt][2 * h + e], p.c2, -mm)) : 0.f;
          split_bf16(x[e], hi[e], lo[e]);
          sum = __fadd_rn(sum, x[e]);
        }
        const int kc = warp * 4 + nb;
        const uint32_t o = static_cast<uint32_t>(pair * kSplit * 2 + ((kc ^ (pair & 7)) << 4) + 4 * tq);
        *reinterpret_cast<uint32_t*>(pt + o) = pack_bf16(hi[0], hi[1]);
        *reinterpret_cast<uint32_t*>(pt_lo + o) = pack_bf16(lo[0], lo[1]);
      }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      if (tq == 0) wsum[warp][pair] = sum;
    }
  cp_async_wait<0>();
  __syncthreads();

  // o = P . V: warp w owns columns 16w .. 16w + 15, one fp32 chain of 16-key
  // steps, hi then lo (steps past every pair's last position add nothing)
  if (warp >= D / 16) return;
  float oc[MT][2][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) oc[mt][nb][i] = 0.f;
  const int vchunk = warp * 2 + (lane >> 4);
  auto load_p = [&](int mt, int kk, uint32_t (&ah)[4], uint32_t (&al)[4]) {
    const int prow = mt * 16 + (lane & 15);
    const int kc = 2 * kk + (lane >> 4);
    const uint32_t o = static_cast<uint32_t>(prow * kSplit * 2 + ((kc ^ (prow & 7)) << 4));
    ldsm_x4(pt_base + o, ah[0], ah[1], ah[2], ah[3]);
    ldsm_x4(pt_lo_base + o, al[0], al[1], al[2], al[3]);
  };
  const int shared_steps = c / 16;  // steps that hold context keys only
#pragma unroll 2
  for (int kk = 0; kk < shared_steps; ++kk) {
    uint32_t b0, b1, b2, b3;
    const int key = kk * 16 + (lane & 15);
    ldsm_x4_t(kv_base + static_cast<uint32_t>(key * D * 2 + ((vchunk ^ (key & 7)) << 4)), b0, b1, b2, b3);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t ah[4], al[4];
      load_p(mt, kk, ah, al);
      mma_bf16_16816(oc[mt][0], ah, b0, b1);
      mma_bf16_16816(oc[mt][1], ah, b2, b3);
      mma_bf16_16816(oc[mt][0], al, b0, b1);
      mma_bf16_16816(oc[mt][1], al, b2, b3);
    }
  }
  for (int kk = shared_steps; kk * 16 < cnt_max; ++kk) {
    const int at = kk * 16 + (lane & 15);  // the position whose V row this lane addresses
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t ah[4], al[4];
      load_p(mt, kk, ah, al);
      for (int i = mt * 16 / G; i < min(nodes, (mt + 1) * 16 / G); ++i) {
        const int depth = at - c + shift;  // of the node's ancestor at this position
        uint32_t addr = zrow_base + (vchunk << 4);
        if (at < c || depth < __popcll(ti.mask[n0 + i])) {
          const int row = at < c ? at : c + paths[i * kTreeMaxNodes + depth];
          addr = kv_base + static_cast<uint32_t>(row * D * 2 + ((vchunk ^ (row & 7)) << 4));
        }
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(addr, b0, b1, b2, b3);
        float tmp[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) tmp[nb][e] = oc[mt][nb][e];
        mma_bf16_16816(tmp[0], ah, b0, b1);
        mma_bf16_16816(tmp[1], ah, b2, b3);
        mma_bf16_16816(tmp[0], al, b0, b1);
        mma_bf16_16816(tmp[1], al, b2, b3);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((mt * 16 + h * 8 + gq) / G == i) {
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
              oc[mt][nb][2 * h] = tmp[nb][2 * h];
              oc[mt][nb][2 * h + 1] = tmp[nb][2 * h + 1];
            }
          }
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (cnt[mt][h] <= 0) continue;
      const int pair = mt * 16 + h * 8 + gq;
      const int64_t base = (static_cast<int64_t>(off + n0 + pair / G) * p.Hq + g * G + pair % G) * p.S + s;
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
        *reinterpret_cast<float2*>(p.ws_o + base * D + warp * 16 + nb * 8 + 2 * tq) =
            make_float2(oc[mt][nb][2 * h], oc[mt][nb][2 * h + 1]);
      if (warp == 0 && tq == 0) {
        float l = wsum[0][pair];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) l = __fadd_rn(l, wsum[w][pair]);
        p.ws_ml[base * 2 + 0] = m[mt][h];
        p.ws_ml[base * 2 + 1] = l;
      }
    }
}

// One block per (query head, node, sequence); thread d folds column d over the
// splits the node sees, with the decode merge's arithmetic.
template <int D>
__global__ void __launch_bounds__(D) attn_tree_merge_kernel(const TreeAttnParams p) {
  __shared__ TreeInfo ti;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, node = blockIdx.y, b = blockIdx.z;
  if (threadIdx.x < 32) tree_load(p.tree, b, ti);
  __syncthreads();
  if (!ti.ok || node >= ti.n) return;
  const int d = threadIdx.x;
  const int64_t row = ti.off + node;
  const int len = ti.ctx + __popcll(ti.mask[node]);
  const int ns = (len + kSplit - 1) / kSplit;
  const int64_t base = (row * p.Hq + h) * p.S;
  float m_acc = -INFINITY, l_acc = 0.f, o_acc = 0.f;
  constexpr int CH = 8;  // partials loaded ahead of the (sequential) fold
  for (int s0 = 0; s0 < ns; s0 += CH) {
    float mv[CH], lv[CH], ov[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (s0 + i < ns) {
        const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + (base + s0 + i) * 2);
        mv[i] = ml.x;
        lv[i] = ml.y;
        ov[i] = p.ws_o[(base + s0 + i) * D + d];
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (s0 + i < ns) {
        const float m_new = fmaxf(m_acc, mv[i]);
        const float a = ex2_approx(__fsub_rn(m_acc, m_new));
        const float c = ex2_approx(__fsub_rn(mv[i], m_new));
        l_acc = __fadd_rn(__fmul_rn(l_acc, a), __fmul_rn(lv[i], c));
        o_acc = __fadd_rn(__fmul_rn(o_acc, a), __fmul_rn(ov[i], c));
        m_acc = m_new;
      }
    }
  }
  p.out[(row * p.Hq + h) * D + d] = __float2bfloat16_rn(__fdiv_rn(o_acc, l_acc));
}

template <int D, int MT>
constexpr size_t split_smem_bytes() {
  return static_cast<size_t>(kSplit + kTreeMaxNodes) * D * 2 + 2 * 16 * MT * kSplit * 2 + D * 2 + 16 * MT * kTreeMaxNodes;
}

template <int D, int MT>
kinv_status launch_split(const TreeAttnParams& p, cudaStream_t stream) {
  void (*kernel)(const TreeAttnParams) = attn_tree_split_kernel<D, MT>;
  const size_t smem = split_smem_bytes<D, MT>();
  const kinv_status attr = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
  if (attr != KINV_OK) return attr;
  const int tiles = (p.tree.max_nodes * p.G + 16 * MT - 1) / (16 * MT);
  return launch_kernel(kernel, dim3(p.Hkv * tiles, p.S, p.tree.B), dim3(kThreads), smem, stream, 1, p);
}

template <int D>
kinv_status launch(const TreeAttnParams& p, cudaStream_t stream) {
  const kinv_status st = p.tree.max_nodes * p.G <= 16 ? launch_split<D, 1>(p, stream) : launch_split<D, 2>(p, stream);
  if (st != KINV_OK) return st;
  return launch_kernel(attn_tree_merge_kernel<D>, dim3(p.Hq, p.tree.max_nodes, p.tree.B), dim3(D), 0, stream, 1, p);
}

size_t tree_workspace_bytes(int64_t rows, int Hq, int D, int S) {
  const size_t o = static_cast<size_t>(rows) * Hq * S * D * 4;
  return ((o + 255) / 256) * 256 + static_cast<size_t>(rows) * Hq * S * 2 * 4;
}

}  // namespace
}  // namespace kinv

using namespace kinv;

extern "C" size_t kinv_attn_tree_workspace(int B, int total_rows, int max_nodes, int Hq, int Hkv, int D,
                                           int max_kv, int split_len) {
  if (B <= 0 || total_rows <= 0 || max_nodes <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_kv <= 0 || split_len <= 0)
    return 0;
  return tree_workspace_bytes(total_rows, Hq, D, static_cast<int>((static_cast<int64_t>(max_kv) + split_len - 1) / split_len));
}

extern "C" kinv_status kinv_attn_tree(const void* q, const void* k_cache, const void* v_cache,
                                      int64_t seq_stride, int64_t tok_stride, const kinv_tree* tree,
                                      void* out, int Hq, int Hkv, int D, int split_len, float scale,
                                      void* workspace, size_t workspace_bytes, kinv_stream stream) {
  const kinv_status st = tree_check(tree);
  if (st != KINV_OK) return st;
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv) return KINV_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != kMaxG) return KINV_ERR_UNSUPPORTED;
  if (D != 64 && D != 128) return KINV_ERR_UNSUPPORTED;
  if (split_len != kSplit) return KINV_ERR_UNSUPPORTED;
  if (tree_empty(tree)) return KINV_OK;
  if (!q || !k_cache || !v_cache || !out || !workspace || tree->max_kv <= 0) return KINV_ERR_INVALID_ARG;
  if (tok_stride < static_cast<int64_t>(Hkv) * D || seq_stride < 0 || (tree->B > 1 && seq_stride == 0))
    return KINV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace) ||
      seq_stride % 8 || tok_stride % 8)
    return KINV_ERR_ALIGNMENT;
  const int64_t S = (static_cast<int64_t>(tree->max_kv) + kSplit - 1) / kSplit;
  if (S > 65535) return KINV_ERR_UNSUPPORTED;
  if (workspace_bytes < tree_workspace_bytes(tree->total_rows, Hq, D, static_cast<int>(S))) return KINV_ERR_WORKSPACE;
  TreeAttnParams p{};
  p.tree = *tree;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k_cache);
  p.v = static_cast<const __nv_bfloat16*>(v_cache);
  p.seq_stride = seq_stride;
  p.tok_stride = tok_stride;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ws_o = static_cast<float*>(workspace);
  const size_t o_bytes = static_cast<size_t>(tree->total_rows) * Hq * S * D * 4;
  p.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + ((o_bytes + 255) / 256) * 256);
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.S = static_cast<int>(S);
  p.c2 = base2_factor(scale, D);
  p.status = device_status_word();
  return D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}
