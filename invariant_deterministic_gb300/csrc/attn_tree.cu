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
#include "attn_tc.cuh"
#include "common.cuh"
#include "tree.cuh"

namespace kinv {
namespace {

constexpr int kSplit = 256;    // keys per split, as in decode and prefill
constexpr int kThreads = 256;  // eight warps, 32 positions each for the softmax
constexpr int kMaxG = 8;
constexpr int kScoreLd = kSplit + 8;
// The splits within the context go to the tcgen05 kernel from this many (sequence, kv
// head, split) triples that the cache may hold times the tree's pairs; trees of at
// most 16 pairs, one MMA tile that the loads bound, with D = 128 and from 512 triples.
// Device time of a call with it / without:
//   D = 128, 16 pairs: 256 triples 16.9 / 14.6 us, 512 23.7 / 24.3, 8,192 184 / 218
//     32 pairs: 128 triples 15.2 / 13.9 us, 256 17.0 / 19.2, 8,192 193 / 307
//     128 pairs: 16 triples 14.1 / 12.8 us, 64 14.8 / 16.6, 2,048 89 / 300
//     256 pairs: 32 triples 15.9 / 25.1 us, 2,048 197 / 813
//   D = 64, 16 pairs: 512 triples 26.1 / 20.2 us, 4,096 99.6 / 89.8
//     33 pairs: 256 triples 21.8 / 29.3 us, 4,096 126 / 220
constexpr int64_t kMinWorkTc = 5120;
constexpr int64_t kMinTriplesTc = 512;

struct TreeAttnParams {
  kinv_tree tree;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t seq_stride, tok_stride;
  __nv_bfloat16* out;
  // Partials, 16 pairs of a (sequence, kv head) side by side: a group's splits
  // follow each other, a split is [D / 8][16 pairs][8].  Group (b, g, i) has
  // index (b * Hkv + g) * groups + i; its pairs are 16 i .. 16 i + 15.
  float* ws_o;    // [B * Hkv * groups][S][D / 8][16][8]
  float* ws_ml;   // [B * Hkv * groups][S][16][2]
  // [B * Hkv * groups], at the first group of each 128 pairs: how many splits
  // their partials of split 0 stand for
  int* ws_cov;
  int groups;
  int Hq, Hkv, G, gs;  // G = Hq / Hkv = 1 << gs
  int S;         // splits per row in the workspace
  float c2;      // fp32(scale * log2 e) > 0
  int tail_only; // the splits that end within the context are another kernel's
  int* status;
};

__device__ __forceinline__ void report_bad_tree(const TreeAttnParams& p) {
  if (threadIdx.x == 0 && p.status) atomicExch(p.status, DEV_TREE_BAD);
}

// Where the partial of a group's split begins, in pairs (rows of D values in
// ws_o, of 2 in ws_ml).
__device__ __forceinline__ int64_t partial_at(const TreeAttnParams& p, int group, int s) {
  return (static_cast<int64_t>(group) * p.S + s) * 16;
}

// A split of a tile of 16 MT pairs of (sequence b, kv head g), by one block.  The
// partial goes to the workspace or, LOCAL, to o_out [16 MT][D] and ml_out [16 MT][2]
// in shared memory (then the tree is loaded whatever the split).
template <int D, int MT, bool LOCAL>
__device__ __forceinline__ void split_block(const TreeAttnParams& p, int g, int tile, int b, int part, TreeInfo& ti,
                                            unsigned char* smem_raw, float* o_out, float* ml_out) {
  constexpr int C8 = D / 8;   // 16-byte chunks per key row
  constexpr int KS = D / 16;  // 16-wide k steps of q . k
  constexpr int R = 16 * MT;  // pairs of the tile
  // scores by position [R][256] fp32 (rows kScoreLd apart: eight rows at one
  // position would share a bank), then P_hi and P_lo [R][256] in their
  // place (8-key chunk kc of row r at chunk kc ^ (r & 7)); a row of zeros; the
  // path of each node of the tile; K, then V (rows of 16-byte chunks, chunk c of
  // row r at chunk c ^ (r & 7)): up to 256 context keys, or up to 255 and the
  // drafted ones
  unsigned char* pt = smem_raw;
  unsigned char* pt_lo = pt + R * kSplit * 2;
  float* scores = reinterpret_cast<float*>(pt);
  unsigned char* zrow = pt + R * kScoreLd * 4;
  unsigned char* paths = zrow + D * 2;  // [R >> gs][64]
  unsigned char* kv = paths + (R >> p.gs) * kTreeMaxNodes;
  __shared__ int depth[kTreeMaxNodes];
  __shared__ float wmax[kThreads / 32][R];
  __shared__ float wsum[kThreads / 32][R];

  int n, ctx, off;
  if (!tree_bounds(p.tree, b, n, ctx, off)) {
    report_bad_tree(p);
    return;
  }
  const int s = (p.tail_only ? ctx / kSplit : 0) + part;
  const int gs = p.gs;  // G = 1 << gs
  const int npt = R >> gs;  // nodes of a tile
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
  // other tiles read the same keys: the default L2 policy keeps them
  auto load = [&](const __nv_bfloat16* src) {
    for (int idx = t; idx < rows * C8; idx += kThreads) {
      const int r = idx / C8, ch = idx % C8;
      const int slot = r < c ? k0 + r : ctx + r - c;
      cp_async16(kv_base + static_cast<uint32_t>(r * D * 2 + ((ch ^ (r & 7)) << 4)),
                 src + seq_off + static_cast<int64_t>(slot) * p.tok_stride + ch * 8);
    }
    cp_async_commit();
  };
  // The tile's q rows first (into the scores' place, chunks swizzled as K's),
  // then the tree, then the long loads: small loads behind K's would wait for it.
  // Row r of the tile is pair r: node n0 + r / G, query head g G + r % G.
  for (int idx = t; idx < (nodes << gs) * C8; idx += kThreads) {
    const int r = idx / C8, ch = idx % C8;
    cp_async16(pt_base + static_cast<uint32_t>(r * D * 2 + ((ch ^ (r & 7)) << 4)),
               p.q + (static_cast<int64_t>(off + n0 + (r >> gs)) * p.Hq + (g << gs) + (r & ((1 << gs) - 1))) * D + ch * 8);
  }
  if (tail || LOCAL) {
    if (warp == 0) {
      tree_load(p.tree, b, ti);
      __syncwarp();
      depth[lane] = __popcll(ti.mask[lane]) - 1;
      depth[lane + 32] = __popcll(ti.mask[lane + 32]) - 1;
    }
    for (int i = t; i < D * 2 / 16; i += kThreads) *reinterpret_cast<uint4*>(zrow + 16 * i) = make_uint4(0, 0, 0, 0);
  }
  load(p.k);
  // V follows into the same buffer once K has been read: towards L2 meanwhile
  for (int idx = t; idx < rows * D / 64; idx += kThreads) {
    const int r = idx / (D / 64), slot = r < c ? k0 + r : ctx + r - c;
    prefetch_l2(p.v + seq_off + static_cast<int64_t>(slot) * p.tok_stride + idx % (D / 64) * 64);
  }
  cp_async_wait<0>();
  __syncthreads();
  if ((tail || LOCAL) && !ti.ok) {
    report_bad_tree(p);
    return;
  }
  if (tail) {
    // the path of a node: the set bits of its mask, ascending
    for (int idx = t; idx < nodes * kTreeMaxNodes; idx += kThreads) {
      const int i = idx / kTreeMaxNodes, j = idx % kTreeMaxNodes;
      if (ti.mask[n0 + i] >> j & 1) paths[i * kTreeMaxNodes + depth[j]] = static_cast<unsigned char>(j);
    }
  }
  // q fragments (A operand): MMA row r of tile mt is pair 16 mt + r (rows of no
  // pair hold anything, and so do their results, which nothing reads)
  uint32_t qa[MT][KS][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int r = mt * 16 + (lane & 15), ch = 2 * ks + (lane >> 4);
      ldsm_x4(pt_base + static_cast<uint32_t>(r * D * 2 + ((ch ^ (r & 7)) << 4)), qa[mt][ks][0], qa[mt][ks][1],
              qa[mt][ks][2], qa[mt][ks][3]);
    }
  __syncthreads();  // the scores take q's place

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
  // warp w: positions 32w + 8nb + 2tq (+1), pairs gq and gq + 8 of each MMA tile
  float sc[4][MT][4];
  int cnt[MT][2];  // positions of this split that the pair sees
  int cnt_max = 0;
  if (!tail) {
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) score_block(warp * 32 + nb * 8, sc[nb]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) cnt[mt][h] = (mt * 16 + h * 8 + gq) >> gs < nodes ? kSplit : 0;
    cnt_max = kSplit;
  } else {
    // every key row's scores, put at the position the key has for the pair
    unsigned long long mask[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = (mt * 16 + h * 8 + gq) >> gs;
        mask[mt][h] = i < nodes ? ti.mask[n0 + i] : 0ull;
        cnt[mt][h] = i < nodes ? max(0, min(kSplit, ctx + depth[n0 + i] + 1 - k0)) : 0;
      }
    for (int blk = warp; blk * 8 < rows; blk += kThreads / 32) {
      float one[MT][4];
      score_block(blk * 8, one);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = blk * 8 + 2 * tq + e, j = key - c;
        int at = key;
        if (j >= 0) at = j < drafted ? c + depth[j] - shift : kSplit;
        if (at < 0 || at >= kSplit || (j >= 0 && at < c)) continue;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (j < 0 || (mask[mt][h] >> j & 1)) scores[(mt * 16 + h * 8 + gq) * kScoreLd + at] = one[mt][2 * h + e];
      }
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* row = scores + (mt * 16 + h * 8 + gq) * kScoreLd + warp * 32 + 2 * tq;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          const float2 v = *reinterpret_cast<const float2*>(row + nb * 8);
          sc[nb][mt][2 * h] = v.x;
          sc[nb][mt][2 * h + 1] = v.y;
        }
      }
    for (int i = 0; i < nodes; ++i) cnt_max = max(cnt_max, min(kSplit, ctx + depth[n0 + i] + 1 - k0));
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
#pragma unroll 4
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
    const int dep = at - c + shift;        // of a node's ancestor at this position
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int i0 = (mt * 16) >> gs, i1 = min(nodes, ((mt + 1) * 16) >> gs);
      if (i0 >= i1) continue;
      uint32_t ah[4], al[4];
      load_p(mt, kk, ah, al);
      float was[2][4];  // the accumulators before this step
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) was[nb][e] = oc[mt][nb][e];
#pragma unroll 2
      for (int i = i0; i < i1; ++i) {
        uint32_t addr = zrow_base + (vchunk << 4);
        if (at < c || dep <= depth[n0 + i]) {
          const int row = at < c ? at : c + paths[i * kTreeMaxNodes + dep];
          addr = kv_base + static_cast<uint32_t>(row * D * 2 + ((vchunk ^ (row & 7)) << 4));
        }
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(addr, b0, b1, b2, b3);
        float tmp[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) tmp[nb][e] = was[nb][e];
        mma_bf16_16816(tmp[0], ah, b0, b1);
        mma_bf16_16816(tmp[1], ah, b2, b3);
        mma_bf16_16816(tmp[0], al, b0, b1);
        mma_bf16_16816(tmp[1], al, b2, b3);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((mt * 16 + h * 8 + gq) >> gs == i) {
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
      const int64_t at = partial_at(p, (b * p.Hkv + g) * p.groups + tile * MT + mt, s);
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
        *reinterpret_cast<float2*>(LOCAL ? o_out + pair * D + warp * 16 + nb * 8 + 2 * tq
                                         : p.ws_o + at * D + ((2 * warp + nb) * 16 + h * 8 + gq) * 8 + 2 * tq) =
            make_float2(oc[mt][nb][2 * h], oc[mt][nb][2 * h + 1]);
      if (warp == 0 && tq == 0) {
        float l = wsum[0][pair];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) l = __fadd_rn(l, wsum[w][pair]);
        *reinterpret_cast<float2*>(LOCAL ? ml_out + pair * 2 : p.ws_ml + (at + h * 8 + gq) * 2) = make_float2(m[mt][h], l);
      }
    }
  if (!LOCAL && s == 0 && t == 0 && tile * R % 128 == 0) p.ws_cov[(b * p.Hkv + g) * p.groups + tile * MT] = 1;
}

// One block per (kv head, tile of 16 MT pairs, split, sequence).
template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 2) attn_tree_split_kernel(const TreeAttnParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ TreeInfo ti;
  pdl_wait();
  pdl_launch_dependents();  // behind the wait: the context kernel starts on what this kernel could
  split_block<D, MT, false>(p, blockIdx.x % p.Hkv, blockIdx.x / p.Hkv, blockIdx.z, blockIdx.y, ti, smem_raw, nullptr, nullptr);
}

// The whole call in one launch where max_kv allows a sequence at most eight splits: a
// cluster of a block per split (block rank s) of a (kv head, tile of 16 pairs,
// sequence); the partials stay in shared memory, and the blocks of the context's
// splits share the tile's pairs and fold them over the cluster in split order,
// with the merge's arithmetic.  Taken while the blocks fit the SMs at two each: a
// block keeps its SM until its cluster is done (4 nodes behind 200 keys, 16 blocks:
// 8.8 us against 10.4 in two launches; 7 small-layer trees behind up to 1,021 keys,
// 140 blocks: 9.6 against 11.4; 64 trees of 4 nodes behind 300 keys, 1,024 blocks:
// 45 against 32).
constexpr int kMaxFused = 8;

template <int D>
__global__ void __launch_bounds__(kThreads, 2) attn_tree_fused_kernel(const TreeAttnParams p) {
  constexpr int W = D / 16;  // columns of a thread in the fold
  extern __shared__ __align__(16) unsigned char smem_raw[];
  float* o_s = reinterpret_cast<float*>(smem_raw);  // [16][D]
  float* ml_s = o_s + 16 * D;                       // [16][2]
  __shared__ TreeInfo ti;
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x, g = blockIdx.y % p.Hkv, tile = blockIdx.y / p.Hkv, b = blockIdx.z;
  split_block<D, 1, true>(p, g, tile, b, s, ti, reinterpret_cast<unsigned char*>(ml_s + 32), o_s, ml_s);
  cluster_sync();
  int n, ctx, off;
  const bool ok = tree_bounds(p.tree, b, n, ctx, off);
  const int owners = ctx / kSplit + 1;  // these blocks loaded the tree
  const int pair = threadIdx.x >> 4, col = (threadIdx.x & 15) * W;
  const int node = ((tile * 16) >> p.gs) + (pair >> p.gs);
  if (ok && s < owners && pair % owners == s && node < n && ti.ok) {
    const int ns = (ctx + __popcll(ti.mask[node]) + kSplit - 1) / kSplit;
    const uint32_t ml_at = smem_addr(ml_s + pair * 2), o_at = smem_addr(o_s + pair * D + col);
    float m_acc = -INFINITY, l_acc = 0.f, o_acc[W];
#pragma unroll
    for (int w = 0; w < W; ++w) o_acc[w] = 0.f;
#pragma unroll 4
    for (int q = 0; q < ns; ++q) {
      const uint32_t ml = map_to_rank(ml_at, q), at = map_to_rank(o_at, q);
      const float m = ld_dsmem_f32(ml), l = ld_dsmem_f32(ml + 4);
      float v[W];
#pragma unroll
      for (int w = 0; w < W; w += 4) {
        const float4 x = ld_dsmem_v4(at + w * 4);
        v[w] = x.x, v[w + 1] = x.y, v[w + 2] = x.z, v[w + 3] = x.w;
      }
      const float m_new = fmaxf(m_acc, m);
      const float a = ex2_approx(__fsub_rn(m_acc, m_new));
      const float c = ex2_approx(__fsub_rn(m, m_new));
      l_acc = __fadd_rn(__fmul_rn(l_acc, a), __fmul_rn(l, c));
#pragma unroll
      for (int w = 0; w < W; ++w) o_acc[w] = __fadd_rn(__fmul_rn(o_acc[w], a), __fmul_rn(v[w], c));
      m_acc = m_new;
    }
    const int64_t head = static_cast<int64_t>(off + node) * p.Hq + (g << p.gs) + (pair & ((1 << p.gs) - 1));
#pragma unroll
    for (int w = 0; w < W; w += 2)
      *reinterpret_cast<uint32_t*>(p.out + head * D + col + w) =
          pack_bf16(__fdiv_rn(o_acc[w], l_acc), __fdiv_rn(o_acc[w + 1], l_acc));
  }
  cluster_sync();  // no block leaves while its partial is read
}

// ---------------------------------------------------------------------------
// The splits that end within the context, on the tcgen05 tensor cores: 128
// pairs of one (sequence, kv head) against 256 keys, the arithmetic of the
// prefill kernel without a mask, each split's (m, l, o) stored as a partial.
//
// A step is (sequence, kv head, split, tile of 128 pairs).  The steps are dealt to
// the blocks (one per SM) in equal runs of T, counted on the device from the
// trees' own numbers.  A block folds the splits that it takes from split 0 on, so
// the order of the steps keeps such beginnings whole.  A chain is a (sequence, kv
// head, tile).  First come the first T splits of every chain that has more and is
// its tree's only tile, a run each; then the chains of at most T splits, one after
// the other (a tree's further tiles read K and V again, which is no more than
// their partials would be, written and read); then the rest, whose splits leave a
// partial each, tiles fastest: a split's further tiles find its K and V in L2.
// Roles (18 warps): warps 0-15 take the softmax, four threads per pair: warp w
// holds TMEM lanes 32 (w % 4) .. + 31 (lane = pair) and keys 64 (w / 4) ..
// + 63 of each split, so a tile's softmax is four warps deep on every
// scheduler; the four exchange raw maxima and 32-key group sums through shared
// memory, in the decode kernel's order.  Warp 16 lane 0 issues the MMAs, warp 17
// lane 0 the TMA loads.
// Tensor memory: three buffers of 128 columns for the scores R of half a split (128
// keys), overwritten 16 keys at a time with their P (packed bf16 pairs: hi in the
// first eight of the 16 columns, lo in the others), then O in D columns.  Half h of
// step i takes buffer (2 i + h) % 3, so the third one receives the first half of
// step i + 1's scores while the softmax of step i runs; the second half follows
// step i's P.V of the first half, which frees its buffer, and then the softmax of
// step i + 1 runs beside step i's P.V of the second half.  The softmax threads read
// step i - 1's O just before they hand over step i's P, and fold or send it behind
// that.  K and V arrive in halves as well, each as soon as the MMAs have read the
// last step's.  (A call with the scores of a step behind the last step's P.V
// and whole K and V tiles / this way: 16 trees of 32 nodes behind up to 32,700 keys
// 304 / 286 us, 64 trees of 1 to 16 behind 2,000 to 4,100 158 / 143, one of 64
// behind 32,000 105 / 100.)
// The fold takes the merge kernel's arithmetic (32 columns of a pair per thread);
// the state of a block's splits is left as the partial of split 0 (ws_cov: how
// many splits that is).
// The partials leave through shared memory and bulk copies: stored straight from
// registers they held up every other shared-memory access of the SM for about
// 2,500 cycles a step (21 - 25 bytes a cycle).
constexpr int kTcSoftmax = 512;  // 16 warps
constexpr int kTcThreads = kTcSoftmax + 64;
constexpr int kTcPairs = 128;
constexpr int kTcBars = 19;
constexpr int kStage = 2048;     // bytes a warp stages at a time: two groups x two 8-column chunks

struct StepCursor {
  int part;                 // 0: beginnings of T splits, 1: whole short chains, 2: the rest
  int b, g, s, tile;
  int off;                  // of the sequence
  int pairs, tiles;
  int lo, splits;           // splits lo .. splits - 1 of a (sequence, kv head) belong to the part
  int T;
};

// Sequence c.b's numbers; returns its steps in c.part, or in all of them.
__device__ __forceinline__ int64_t cursor_load(const TreeAttnParams& p, StepCursor& c, bool all = false) {
  int n, ctx;
  c.lo = c.splits = c.tiles = 0;
  if (!tree_bounds(p.tree, c.b, n, ctx, c.off)) return 0;
  c.pairs = n << p.gs;
  c.tiles = (c.pairs + kTcPairs - 1) / kTcPairs;
  const int splits = ctx / kSplit;
  if (all)
    c.splits = splits;
  else if (splits <= c.T)
    c.splits = c.part == 1 ? splits : 0;
  else if (c.tiles > 1)
    c.splits = c.part == 2 ? splits : 0;
  else if (c.part != 1)
    c.lo = c.part == 2 ? c.T : 0, c.splits = c.part == 2 ? splits : c.T;
  return static_cast<int64_t>(p.Hkv) * (c.splits - c.lo) * c.tiles;
}
// The next step; whether its rows are others.
__device__ __forceinline__ bool cursor_next(const TreeAttnParams& p, StepCursor& c) {
  if (c.part == 2) {
    if (++c.tile < c.tiles) return true;
    c.tile = 0;
    if (++c.s < c.splits) return c.tiles > 1;
  } else {
    if (++c.s < c.splits) return false;
    c.s = c.lo;
    if (++c.tile < c.tiles) return true;
    c.tile = 0;
  }
  if (++c.g >= p.Hkv) {
    c.g = 0;
    do {
      if (++c.b >= p.tree.B) {
        c.b = 0;
        ++c.part;
      }
    } while (c.part < 3 && cursor_load(p, c) == 0);
  }
  c.s = c.lo;
  return true;
}

// This block's run of steps, by one warp: cursor at its first and its length.
__device__ __forceinline__ void cursor_start(const TreeAttnParams& p, StepCursor& out, int& count) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0;
  StepCursor c;
  c.part = c.T = 0;
  for (c.b = lane; c.b < p.tree.B; c.b += 32) total += cursor_load(p, c, true);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int64_t T = (total + gridDim.x - 1) / gridDim.x;  // (far below 2^31 for any cache that memory holds)
  const int64_t u0 = min(total, T * blockIdx.x), u1 = min(total, u0 + T);
  if (lane == 0) count = static_cast<int>(u1 - u0);
  if (u1 == u0) return;
  c.T = static_cast<int>(T);
  int64_t before = 0;
  for (c.part = 0; c.part < 3; ++c.part) {
    for (int b0 = 0; b0 < p.tree.B; b0 += 32) {
      c.b = b0 + lane;
      const int64_t mine = c.b < p.tree.B ? cursor_load(p, c) : 0;
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const bool here = before + incl - mine <= u0 && u0 < before + incl;
      if (here) {
        const int64_t u = u0 - (before + incl - mine);
        const int splits = c.splits - c.lo;
        c.tile = static_cast<int>(c.part == 2 ? u % c.tiles : u / splits % c.tiles);
        c.s = c.lo + static_cast<int>(c.part == 2 ? u / c.tiles % splits : u % splits);
        c.g = static_cast<int>(u / c.tiles / splits);
        out = c;
      }
      if (__any_sync(0xffffffffu, here)) return;
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
}

// Whether the barrier's phase of this parity is complete; never waits.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// x - h, exactly: the mixed-precision fma takes the bf16 halves as they are (the
// softmax's arithmetic alone, 256 keys by 128 pairs: 1,545 cycles an SM; 1,856 with
// the halves widened first).
__device__ __forceinline__ float2 less_bf16(float2 x, __nv_bfloat162 h) {
  float2 r;
  asm("{\n\t.reg .b16 a, b, m;\n\tmov.b32 {a, b}, %2;\n\tmov.b16 m, 0xBF80;\n\t"
      "fma.rn.f32.bf16 %0, a, m, %3;\n\tfma.rn.f32.bf16 %1, b, m, %4;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(*reinterpret_cast<const uint32_t*>(&h)), "f"(x.x), "f"(x.y));
  return r;
}

// An asynchronous copy of `bytes` (a multiple of 16) from shared to global
// memory, in this thread's current bulk group.
__device__ __forceinline__ void bulk_store(float* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Waits until this thread's copies have read their source / are complete.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tree_ctx_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const TreeAttnParams p) {
  constexpr int DS = D / 64;                // 64-wide slices of the head dimension
  constexpr int Q_SLICE = kTcPairs * 128;   // [128 pairs][64]
  constexpr int Q_BYTES = DS * Q_SLICE;
  constexpr int KV_SLICE = kSplit * 128;    // [256 keys][64]
  constexpr int KV_BYTES = DS * KV_SLICE;
  constexpr int HALF = KV_SLICE / 2;        // 128 keys of a slice
  constexpr uint32_t O_COL = 384;
  constexpr int DQ = D / 4;                 // output columns per softmax thread
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* q_s = base;
  unsigned char* k_s = q_s + Q_BYTES;
  unsigned char* v_s = k_s + KV_BYTES;
  unsigned char* stage = v_s + KV_BYTES;    // [16 warps][2 groups][2 chunks][16 pairs][8] fp32
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage + 16 * kStage);
  float* x_max = reinterpret_cast<float*>(bars + kTcBars + 1);  // [4][128] raw maxima
  float* x_sum = x_max + 4 * kTcPairs;                          // [8][128] 32-key group sums
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ StepCursor start;
  __shared__ StepCursor chains[16];  // of each softmax warp, advanced where its chain ends
  __shared__ int count_s;
  auto k_full = [&](int h) { return smem_addr(bars + 0 + h); };    // of keys 128 h ..
  auto k_empty = [&](int h) { return smem_addr(bars + 2 + h); };
  auto v_full = [&](int h) { return smem_addr(bars + 4 + h); };
  auto v_empty = [&](int h) { return smem_addr(bars + 6 + h); };
  // R of keys 128 h .. written; two of each, as step i + 1's may be before every
  // thread has seen step i's
  auto s_full = [&](int i, int h) { return smem_addr(bars + 8 + 2 * (i & 1) + h); };
  auto p_full = [&](int j) { return smem_addr(bars + 12 + j); };   // P chunk j written
  const uint32_t o_full = smem_addr(bars + 16), o_empty = smem_addr(bars + 17), done_bar = smem_addr(bars + 18);

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  // No wait here: the kernel before this one is the tail's, which touches nothing that
  // this one does, and every one of its blocks lets this one start only behind its own
  // wait.  So all before the tail is complete when a block of this kernel runs: the
  // writers of q, the caches and the tree, and the merge of an earlier call, which read
  // the partials that this one overwrites.  The wait stands at the end, as what follows
  // needs both.  (No early launch of the merge: its
  // blocks beside these cost 25 us of 130 at 64 nodes behind 32,000 keys.)
  if (warp == 0) cursor_start(p, start, count_s);
  __syncthreads();
  const int count = count_s;
  if (count == 0) {
    pdl_wait();
    return;
  }
  if (t == 0) {
    for (int i = 0; i < kTcBars; ++i) {
      // p_full: the 128 threads of its chunk; o_empty: every softmax thread
      const int arrivals = (i >= 12 && i < 16) ? kTcPairs : i == 17 ? kTcSoftmax : 1;
      mbar_init(smem_addr(bars + i), arrivals);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 16) tmem_alloc(smem_addr(&tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  int* status = p.status;

  if (warp == 17) {
    // ---- TMA: the halves of K (and its Q, where that is another) and V, in the
    // order in which the MMAs give their places up
    if (lane == 0) {
      StepCursor c = start;
      const uint64_t q_pol = l2_policy_evict_last();
      const uint64_t kv_pol = l2_policy_evict_first();
      int vb, vg, vs;  // the step whose V is next
      uint64_t v_pol;
      // keys that another tile is about to read should stay in L2
      auto pol = [&]() { return c.tile + 1 < c.tiles ? q_pol : kv_pol; };
      auto v_is_next = [&]() { vb = c.b, vg = c.g, vs = c.s, v_pol = pol(); };
      auto load_q = [&]() {
        for (int ds = 0; ds < DS; ++ds)
          tma_load_3d(smem_addr(q_s + ds * Q_SLICE), &tmQ, 64 * ds, c.g << p.gs, c.off + (c.tile * kTcPairs >> p.gs),
                      k_full(0), q_pol);
      };
      auto load_k = [&](int h, bool new_q) {
        mbar_arrive_expect_tx(k_full(h), DS * HALF + (new_q ? Q_BYTES : 0));
        for (int ds = 0; ds < DS; ++ds)
          tma_load_4d(smem_addr(k_s + ds * KV_SLICE + h * HALF), &tmK, 64 * ds, c.g, c.s * kSplit + 128 * h, c.b,
                      k_full(h), pol());
      };
      auto load_v = [&](int h) {
        mbar_arrive_expect_tx(v_full(h), DS * HALF);
        for (int ds = 0; ds < DS; ++ds)
          tma_load_4d(smem_addr(v_s + ds * KV_SLICE + h * HALF), &tmV, 64 * ds, vg, vs * kSplit + 128 * h, vb,
                      v_full(h), v_pol);
      };
      load_k(0, true);
      load_q();
      load_k(1, false);
      v_is_next();
      load_v(0);
      load_v(1);
      int k_issued[2] = {1, 1}, v_issued[2] = {1, 1};
      bool ok = true;
      for (int n = 1; n <= count && ok; ++n) {  // K of step n, V of step n - 1
        const bool new_q = n < count && cursor_next(p, c);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (ok && n < count) {
            ok = !abort_flag && mbar_wait_bounded(k_empty(h), (n - 1) & 1, status, DEV_TIMEOUT_ATTN);
            if (ok) {
              if (h == 1 && new_q) load_q();  // the last scores that read Q are done
              load_k(h, h == 0 && new_q);
              ++k_issued[h];
            }
          }
          if (ok && n >= 2) {
            ok = !abort_flag && mbar_wait_bounded(v_empty(h), n & 1, status, DEV_TIMEOUT_ATTN);
            if (ok) {
              load_v(h);
              ++v_issued[h];
            }
          }
        }
        v_is_next();
      }
      if (!ok) abort_flag = 1;
      // loads still in flight (only after an abort) land before the block exits
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mbar_wait_bounded(k_full(h), (k_issued[h] - 1) & 1, nullptr, 0);
        mbar_wait_bounded(v_full(h), (v_issued[h] - 1) & 1, nullptr, 0);
      }
    }
    __syncwarp();
  } else if (warp == 16) {
    // ---- MMA issue
    if (lane == 0) {
      constexpr uint32_t idesc_r = tc_idesc(128, 0);
      constexpr uint32_t idesc_o = tc_idesc(D, 1);
      const uint64_t qd = desc_k_sw128(smem_addr(q_s)), kd = desc_k_sw128(smem_addr(k_s));
      const uint64_t vd = desc_mn_sw128(smem_addr(v_s), KV_SLICE);
      bool ok = true;
      auto wait = [&](uint32_t bar, int phase) {
        ok = ok && !abort_flag && mbar_wait_bounded(bar, phase & 1, status, DEV_TIMEOUT_ATTN);
        return ok;
      };
      // step i's scores of keys 128 h .., whose K is there
      auto scores = [&](int i, int h) {
        tc_fence_after();
        const uint32_t col = tmem + static_cast<uint32_t>((2 * i + h) % 3 * 128);
#pragma unroll
        for (int ds = 0; ds < DS; ++ds)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(col, qd + static_cast<uint64_t>((ds * Q_SLICE + kk * 32) >> 4),
                      kd + static_cast<uint64_t>((ds * KV_SLICE + h * HALF + kk * 32) >> 4), idesc_r,
                      (ds | kk) != 0 ? 1u : 0u);
        umma_commit(s_full(i, h));
        umma_commit(k_empty(h));
      };
      // step i's P.V of chunks 2h and 2h + 1
      auto weighted = [&](int i, int h) {
        if (!wait(v_full(h), i)) return;
        const uint32_t p_col = tmem + static_cast<uint32_t>((2 * i + h) % 3 * 128);
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          if (!wait(p_full(2 * h + jj), i)) return;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t vdesc = vd + static_cast<uint64_t>(((8 * h + 4 * jj + kk) * 2048) >> 4);
            const uint32_t p_hi = p_col + static_cast<uint32_t>(64 * jj + 16 * kk);
            umma_bf16_tmem_a(tmem + O_COL, p_hi, vdesc, idesc_o, (h | jj | kk) != 0 ? 1u : 0u);
            umma_bf16_tmem_a(tmem + O_COL, p_hi + 8, vdesc, idesc_o, 1u);
          }
        }
        umma_commit(v_empty(h));
        if (h == 1) umma_commit(o_full);
      };
      if (wait(k_full(0), 0)) scores(0, 0);
      if (wait(k_full(1), 0)) scores(0, 1);
      for (int i = 0; i < count && ok; ++i) {
        const bool more = i + 1 < count;
        int next = 0;  // halves of step i + 1's scores issued
        auto try_scores = [&]() {
          if (more && next < 2 && mbar_test(k_full(next), (i + 1) & 1)) scores(i + 1, next++);
        };
        // the first half's where its K comes before step i's P
        if (more) {
          const unsigned long long t0 = globaltimer_ns();
          while (next == 0 && !mbar_test(p_full(0), i & 1)) {
            try_scores();
            if (abort_flag || globaltimer_ns() - t0 > kWaitLimitNs) break;
          }
        }
        if (i > 0 && !wait(o_empty, i - 1)) break;
        weighted(i, 0);
        if (!ok) break;
        if (next == 0) try_scores();
        if (next == 1) try_scores();
        weighted(i, 1);
        for (; more && next < 2 && wait(k_full(next), i + 1);) scores(i + 1, next++);
      }
      if (!ok) abort_flag = 1;
      umma_commit(done_bar);
      mbar_wait_bounded(done_bar, 0, status, DEV_TIMEOUT_ATTN);
    }
    __syncwarp();
  } else {
    // ---- four threads per pair
    const int quad = warp & 3, j = warp >> 2;  // lanes 32 quad .., keys 64 j .. and output columns D/4 j ..
    const int pr = quad * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t slot = smem_addr(stage) + warp * kStage;
    const float c2 = p.c2;
    bool ok = true;
    auto quad_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + quad) : "memory"); };
    // the quadrant's barrier, returning whether `v` holds for any of its threads
    auto quad_sync_or = [&](bool v) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
          "bar.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(r)
          : "r"(static_cast<uint32_t>(v)), "r"(1 + quad)
          : "memory");
      return r != 0;
    };
    auto check = [&](bool waited) {
      if (__any_sync(0xffffffffu, !waited || abort_flag)) {
        abort_flag = 1;
        ok = false;
      }
    };
    // sends D/4 columns of 32 pairs, this thread's in v, to the partial at `at`
    // (that of the first of the warp's two groups; `second`: the other has pairs)
    auto send = [&](const uint32_t (&v)[DQ], int64_t at, bool second) {
#pragma unroll
      for (int k0 = 0; k0 < DQ / 8; k0 += 2) {
        if (lane == 0) bulk_wait_read();  // the last copies have read the stage
        __syncwarp();
#pragma unroll
        for (int k = k0; k < k0 + 2; ++k) {
          const uint32_t dst = slot + (lane >> 4) * 1024 + (k - k0) * 512 + (lane & 15) * 32;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v[8 * k]), "r"(v[8 * k + 1]),
                       "r"(v[8 * k + 2]), "r"(v[8 * k + 3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 16), "r"(v[8 * k + 4]), "r"(v[8 * k + 5]),
                       "r"(v[8 * k + 6]), "r"(v[8 * k + 7])
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          float* dst = p.ws_o + at * D + (j * (DQ / 8) + k0) * 128;
          bulk_store(dst, slot, 1024);
          if (second) bulk_store(dst + static_cast<int64_t>(p.S) * 16 * D, slot + 1024, 1024);
          bulk_commit();
        }
      }
    };
    // the state of the splits folded so far (l of the first quarter's threads only)
    float o_acc[DQ], m_acc = 0.f, l_acc = 0.f;
    // what the last step left: its place, live pairs and statistics, whether it
    // is folded, and (end_prev) whether the state is complete with it
    int group_prev = 0, s_prev = 0, live_prev = 0;
    float m_prev = 0.f, l_prev = 0.f;
    bool fold_prev = false, end_prev = false;
    // step i's O out of tensor memory
    auto read_o = [&](int i, uint32_t (&v)[DQ]) {
      check(mbar_wait_bounded(o_full, i & 1, status, DEV_TIMEOUT_ATTN));
      tc_fence_after();
      if constexpr (DQ == 32)
        tmem_ld32(lane_base + O_COL + static_cast<uint32_t>(j * DQ), v);
      else
        tmem_ld16(lane_base + O_COL + static_cast<uint32_t>(j * DQ), v);
      tc_fence_before();
      mbar_arrive(o_empty);
    };
    // folds it, or sends it as a partial
    auto take_o = [&](uint32_t (&v)[DQ]) {
      if (live_prev > 0) {
        if (!fold_prev) {
          send(v, partial_at(p, group_prev, s_prev), live_prev > 16);
        } else if (s_prev == 0) {
          // the merge's first step: 0 * 0 + x * 1
          m_acc = m_prev;
          l_acc = __fadd_rn(0.f, l_prev);
#pragma unroll
          for (int d = 0; d < DQ; ++d) o_acc[d] = __fadd_rn(0.f, __uint_as_float(v[d]));
        } else {
          const float m_new = fmaxf(m_acc, m_prev);
          const float a = ex2_approx(__fsub_rn(m_acc, m_new));
          const float c = ex2_approx(__fsub_rn(m_prev, m_new));
          l_acc = __fadd_rn(__fmul_rn(l_acc, a), __fmul_rn(l_prev, c));
#pragma unroll
          for (int d = 0; d < DQ; ++d)
            o_acc[d] = __fadd_rn(__fmul_rn(o_acc[d], a), __fmul_rn(__uint_as_float(v[d]), c));
          m_acc = m_new;
        }
      }
      if (fold_prev && end_prev && ok) {  // the state as the partial of split 0
        if (live_prev > 0) {
          const int64_t at = partial_at(p, group_prev, 0);
#pragma unroll
          for (int d = 0; d < DQ; ++d) v[d] = __float_as_uint(o_acc[d]);
          send(v, at, live_prev > 16);
          if (j == 0 && lane < live_prev)
            *reinterpret_cast<float2*>(p.ws_ml + (at + (lane >> 4) * (static_cast<int64_t>(p.S) * 16) + (lane & 15)) * 2) =
                make_float2(m_acc, l_acc);
        }
        if (warp == 0 && lane == 0) p.ws_cov[group_prev] = s_prev + 1;
      }
    };
    // the chain: its last step, this warp's live pairs (the same for the
    // quadrant's four warps) and first group, whether this block folds it
    int s, end, live, group;
    bool folding;
    auto begin_chain = [&](const StepCursor& c) {
      s = c.s;
      end = c.part == 2 && c.tiles > 1 ? s + 1 : c.splits;
      folding = s == 0;
      live = min(32, c.pairs - c.tile * kTcPairs - quad * 32);
      group = (c.b * p.Hkv + c.g) * p.groups + c.tile * (kTcPairs / 16) + quad * 2;
    };
    begin_chain(start);
    if (lane == 0) chains[warp] = start;
    __syncwarp();
    for (int i = 0; i < count; ++i) {
      check(mbar_wait_bounded(s_full(i, j >> 1), (i >> 1) & 1, status, DEV_TIMEOUT_ATTN));
      tc_fence_after();
      const uint32_t r_col = lane_base + static_cast<uint32_t>((2 * i + (j >> 1)) % 3 * 128 + (j & 1) * 64);
      if (live > 0) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
          tmem_ld32(r_col + 32 * h, v);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            mx[0] = fmax3(mx[0], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            mx[1] = fmax3(mx[1], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
          }
        }
        x_max[j * kTcPairs + pr] = fmaxf(mx[0], mx[1]);
      }
      // one decision for the quadrant's 128 threads: leave if any has given up
      if (quad_sync_or(!ok || abort_flag)) {
        ok = false;
        break;
      }
      float m = 0.f, l = 0.f;
      if (live > 0) {
        m = __fmul_rn(fmaxf(fmaxf(x_max[pr], x_max[kTcPairs + pr]), fmaxf(x_max[2 * kTcPairs + pr], x_max[3 * kTcPairs + pr])), c2);
        const float2 c2x2 = make_float2(c2, c2), neg_m2 = make_float2(-m, -m);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // l in the decode kernel's order: key 8nb + 2tq + e into partial tq
          // in (nb, e) order, then (0 + 1) + (2 + 3)
          float sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t col = r_col + 32 * h + 16 * half;
            uint32_t v[16], hp[8], lp[8];  // bf16 pairs of the high and the low halves
            tmem_ld16(col, v);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 arg = __ffma2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2x2, neg_m2);
              const float2 x = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));
              const __nv_bfloat162 h2 = __float22bfloat162_rn(x);
              const __nv_bfloat162 l2 = __float22bfloat162_rn(less_bf16(x, h2));
              hp[e / 2] = *reinterpret_cast<const uint32_t*>(&h2);
              lp[e / 2] = *reinterpret_cast<const uint32_t*>(&l2);
              sq[e / 2 % 4] = __fadd_rn(__fadd_rn(sq[e / 2 % 4], x.x), x.y);
            }
            tmem_st8(col, hp);
            tmem_st8(col + 8, lp);
          }
          x_sum[(2 * j + h) * kTcPairs + pr] = __fadd_rn(__fadd_rn(sq[0], sq[1]), __fadd_rn(sq[2], sq[3]));
        }
        tmem_st_wait();
      }
      if (i > 0) {
        uint32_t o[DQ];
        read_o(i - 1, o);
        mbar_arrive(p_full(j));
        take_o(o);
      } else {
        tc_fence_before();
        mbar_arrive(p_full(j));
      }
      quad_sync();
      if (j == 0 && lane < live) {
        l = x_sum[pr];
#pragma unroll
        for (int q = 1; q < 8; ++q) l = __fadd_rn(l, x_sum[q * kTcPairs + pr]);
        if (!folding)
          *reinterpret_cast<float2*>(p.ws_ml + (partial_at(p, group, s) + (lane >> 4) * (static_cast<int64_t>(p.S) * 16) + (lane & 15)) * 2) =
              make_float2(m, l);
      }
      group_prev = group;
      s_prev = s;
      live_prev = live;
      m_prev = m;
      l_prev = l;
      fold_prev = folding;
      ++s;
      end_prev = s == end || i + 1 == count;
      if (s == end && i + 1 < count) {
        if (lane == 0) {
          StepCursor c = chains[warp];
          c.s = s - 1;
          cursor_next(p, c);
          chains[warp] = c;
        }
        __syncwarp();
        begin_chain(chains[warp]);
        __syncwarp();
      }
    }
    if (ok) {
      uint32_t o[DQ];
      read_o(count - 1, o);
      if (ok) take_o(o);
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  pdl_wait();
}

// Folds the splits that each node sees, with the decode merge's arithmetic.  A
// block takes 16 pairs of a (sequence, kv head) and 32 columns, a warp eight of
// them: a lane half of those for one pair, so a warp's loads of a split are 512
// contiguous bytes.  The first partials are requested before the tree is read: a
// node of any depth sees the splits up to position ctx_len.  A fold runs CH partials
// behind its loads: six while blocks fill the SMs eight deep, sixteen where four per
// SM are all there are (a call for 64 nodes behind 32,000 keys, 512 blocks: 98 us
// with six, 91 with sixteen; 64 trees of 1 to 16 nodes, 8,192 blocks: 140 and 150).
constexpr int kMergePairs = 16;
constexpr int kMergeThreads = 128;

template <int D, int CH>
__global__ void __launch_bounds__(kMergeThreads, CH > 6 ? 4 : 8) attn_tree_merge_kernel(const TreeAttnParams p) {
  __shared__ TreeInfo ti;
  pdl_launch_dependents();
  pdl_wait();
  constexpr int QUARTERS = D / 32;
  const int lane = threadIdx.x & 31;
  const int k = static_cast<int>(blockIdx.x) % QUARTERS * 4 + (threadIdx.x >> 5);
  const int pair0 = static_cast<int>(blockIdx.x) / QUARTERS * kMergePairs;
  const int g = blockIdx.y, b = blockIdx.z;
  const int pair = pair0 + (lane >> 1);
  int n, ctx, off;
  if (!tree_bounds(p.tree, b, n, ctx, off) || pair0 >= n << p.gs) return;
  const bool live = pair < n << p.gs;
  const int group = (b * p.Hkv + g) * p.groups + (pair0 >> 4);
  const int64_t at = partial_at(p, group, 0) + (lane >> 1);
  const float* ml_at = p.ws_ml + at * 2;
  const float* o_at = p.ws_o + partial_at(p, group, 0) * D + (k * 16 + (lane >> 1)) * 8 + (lane & 1) * 4;
  // partial q of the fold: 0 stands for the first cov splits, the others for one
  // each (clamped: the count of a tree that is left out was never written)
  const int cov = max(1, min(p.ws_cov[group - (pair0 >> 4) % 8], ctx / kSplit));
  float2 ml[CH];
  float4 o[CH];
  auto load = [&](int q0, int nq) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (q0 + i >= nq) continue;
      const int s = q0 + i == 0 ? 0 : cov - 1 + q0 + i;
      ml[i] = *reinterpret_cast<const float2*>(ml_at + static_cast<int64_t>(s) * 32);
      o[i] = *reinterpret_cast<const float4*>(o_at + static_cast<int64_t>(s) * (16 * D));
    }
  };
  const int sure = ctx / kSplit + 2 - cov;  // partials that every node sees
  load(0, sure);
  if (threadIdx.x < 32) tree_load(p.tree, b, ti);
  __syncthreads();
  if (!ti.ok || !live) return;
  const int node = pair >> p.gs;
  const int nq = (ctx + __popcll(ti.mask[node]) + kSplit - 1) / kSplit + 1 - cov;
  float m_acc = -INFINITY, l_acc = 0.f;
  float4 o_acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int q0 = 0; q0 < nq; q0 += CH) {
    if (q0 > 0 || (sure < CH && nq > sure)) load(q0, nq);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (q0 + i < nq) {
        const float m_new = fmaxf(m_acc, ml[i].x);
        const float a = ex2_approx(__fsub_rn(m_acc, m_new));
        const float c = ex2_approx(__fsub_rn(ml[i].x, m_new));
        l_acc = __fadd_rn(__fmul_rn(l_acc, a), __fmul_rn(ml[i].y, c));
        o_acc.x = __fadd_rn(__fmul_rn(o_acc.x, a), __fmul_rn(o[i].x, c));
        o_acc.y = __fadd_rn(__fmul_rn(o_acc.y, a), __fmul_rn(o[i].y, c));
        o_acc.z = __fadd_rn(__fmul_rn(o_acc.z, a), __fmul_rn(o[i].z, c));
        o_acc.w = __fadd_rn(__fmul_rn(o_acc.w, a), __fmul_rn(o[i].w, c));
        m_acc = m_new;
      }
    }
  }
  const int64_t head = static_cast<int64_t>(off + node) * p.Hq + (g << p.gs) + (pair & ((1 << p.gs) - 1));
  *reinterpret_cast<uint2*>(p.out + head * D + 8 * k + (lane & 1) * 4) =
      make_uint2(pack_bf16(__fdiv_rn(o_acc.x, l_acc), __fdiv_rn(o_acc.y, l_acc)),
                 pack_bf16(__fdiv_rn(o_acc.z, l_acc), __fdiv_rn(o_acc.w, l_acc)));
}

template <int D, int MT>
size_t split_smem_bytes(const TreeAttnParams& p) {
  // 256 key rows, or up to 255 and the drafted ones; scores are taken eight rows at a time
  const int kv_rows = kSplit + (p.tree.max_nodes + 7) / 8 * 8;
  return 16 * MT * kScoreLd * 4 + D * 2 + (16 * MT / p.G) * kTreeMaxNodes + static_cast<size_t>(kv_rows) * D * 2;
}

template <int D, int MT>
kinv_status launch_split(const TreeAttnParams& p, cudaStream_t stream) {
  void (*kernel)(const TreeAttnParams) = attn_tree_split_kernel<D, MT>;
  const size_t smem = split_smem_bytes<D, MT>(p);
  const kinv_status attr = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
  if (attr != KINV_OK) return attr;
  const int tiles = (p.tree.max_nodes * p.G + 16 * MT - 1) / (16 * MT);
  const int splits = p.tail_only ? (p.S < 2 ? p.S : 2) : p.S;
  return launch_kernel(kernel, dim3(p.Hkv * tiles, splits, p.tree.B), dim3(kThreads), smem, stream, 1, p);
}

template <int D>
kinv_status launch_fused(const TreeAttnParams& p, cudaStream_t stream) {
  const size_t smem = 16 * D * 4 + 32 * 4 + split_smem_bytes<D, 1>(p);
  const kinv_status attr = ensure_smem(reinterpret_cast<const void*>(attn_tree_fused_kernel<D>), smem);
  if (attr != KINV_OK) return attr;
  const int tiles = (p.tree.max_nodes * p.G + 15) / 16;
  return launch_kernel(attn_tree_fused_kernel<D>, dim3(p.S, p.Hkv * tiles, p.tree.B), dim3(kThreads), smem, stream, p.S, p);
}

template <int D>
constexpr size_t ctx_smem_bytes() {
  return 1024 + static_cast<size_t>(D / 64) * kTcPairs * 128 + 2 * static_cast<size_t>(D / 64) * kSplit * 128 +
         16 * kStage + (kTcBars + 1) * 8 + 12 * kTcPairs * 4;
}

// The tensor maps of the context kernel; false where a stride or size is
// outside what a map can describe.
template <int D>
bool encode_maps(const TreeAttnParams& p, CUtensorMap* mq, CUtensorMap* mk, CUtensorMap* mv) {
  const uint64_t qd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(p.Hq), static_cast<uint64_t>(p.tree.total_rows)};
  const uint64_t qs[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(p.Hq) * D * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(p.G), static_cast<uint32_t>(kTcPairs / p.G)};
  const uint64_t kd[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(p.Hkv), static_cast<uint64_t>(p.tree.max_kv),
                          static_cast<uint64_t>(p.tree.B)};
  // one sequence: any sequence stride describes it (the coordinate is 0)
  const int64_t sst = p.tree.B > 1 ? p.seq_stride : static_cast<int64_t>(p.tree.max_kv) * p.tok_stride;
  const uint64_t ks[3] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(p.tok_stride) * 2, static_cast<uint64_t>(sst) * 2};
  const uint32_t kb[4] = {64, 1, static_cast<uint32_t>(kSplit / 2), 1};
  return encode_map(mq, p.q, 3, qd, qs, qb) && encode_map(mk, p.k, 4, kd, ks, kb) && encode_map(mv, p.v, 4, kd, ks, kb);
}

template <int D>
kinv_status launch(TreeAttnParams p, cudaStream_t stream) {
  const size_t smem = ctx_smem_bytes<D>();
  const int sms = sm_count();
  CUtensorMap mq, mk, mv;
  const int pairs = p.tree.max_nodes * p.G;
  const int64_t triples = static_cast<int64_t>(p.tree.B) * p.Hkv * (p.tree.max_kv / kSplit);
  p.tail_only = (pairs > 16 ? triples * pairs >= kMinWorkTc : D == 128 && triples >= kMinTriplesTc) &&
                smem <= static_cast<size_t>(max_smem_optin()) && encode_maps<D>(p, &mq, &mk, &mv);
  // tiles of 16 pairs where they are the whole tree, where tiles of 32 would leave
  // SMs without a block, and where two blocks with tiles of 32 (and 3 KB of
  // statistics) do not fit an SM (8 trees of 64 nodes behind 300 keys: 48 us a
  // call against 53; with 32 nodes, where they fit, 33 against 28)
  const bool small = pairs <= 16 ||
                     static_cast<int64_t>(p.tree.B) * p.Hkv * ((pairs + 31) / 32) * (p.tail_only ? 1 : p.S) < sms ||
                     2 * (split_smem_bytes<D, 2>(p) + 3 * 1024 + smem_reserved_per_block()) > static_cast<size_t>(smem_per_sm());
  if (small && !p.tail_only && p.S <= kMaxFused &&
      static_cast<int64_t>(p.tree.B) * p.Hkv * ((pairs + 15) / 16) * p.S <= 2 * sms)
    return launch_fused<D>(p, stream);
  kinv_status st = small ? launch_split<D, 1>(p, stream) : launch_split<D, 2>(p, stream);
  if (st != KINV_OK) return st;
  if (p.tail_only) {
    void (*kernel)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const TreeAttnParams) = attn_tree_ctx_kernel<D>;
    st = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
    if (st != KINV_OK) return st;
    st = launch_kernel(kernel, dim3(sms), dim3(kTcThreads), smem, stream, 1, mq, mk, mv, p);
    if (st != KINV_OK) return st;
  }
  const dim3 grid((pairs + kMergePairs - 1) / kMergePairs * (D / 32), p.Hkv, p.tree.B);
  const bool deep = static_cast<int64_t>(grid.x) * grid.y * grid.z <= 4 * sms;
  return launch_kernel(deep ? attn_tree_merge_kernel<D, 16> : attn_tree_merge_kernel<D, 6>, grid, dim3(kMergeThreads), 0,
                       stream, 1, p);
}

// The workspace: partials (on a 256-byte boundary), their statistics, ws_cov.
struct TreeWorkspace {
  int64_t groups, pairs;  // groups of a kv head; rows of D values in all
  size_t o, ml, cov, bytes;
  TreeWorkspace(int64_t B, int max_nodes, int Hq, int Hkv, int D, int64_t S) {
    groups = (static_cast<int64_t>(max_nodes) * (Hq / Hkv) + 15) / 16;
    pairs = B * Hkv * groups * S * 16;
    o = 0;
    ml = o + static_cast<size_t>(pairs) * D * 4;
    cov = ml + static_cast<size_t>(pairs) * 8;
    bytes = 256 + cov + static_cast<size_t>(B * Hkv * groups) * 4;  // 256 to align the base
  }
};

}  // namespace
}  // namespace kinv

using namespace kinv;

extern "C" size_t kinv_attn_tree_workspace(int B, int total_rows, int max_nodes, int Hq, int Hkv, int D,
                                           int max_kv, int split_len) {
  if (B <= 0 || total_rows <= 0 || max_nodes <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_kv <= 0 || split_len <= 0)
    return 0;
  return TreeWorkspace(B, max_nodes, Hq, Hkv, D, (static_cast<int64_t>(max_kv) + split_len - 1) / split_len).bytes;
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
  const TreeWorkspace w(tree->B, tree->max_nodes, Hq, Hkv, D, S);
  if (static_cast<int64_t>(tree->B) * Hkv * w.groups > 0x7fffffff) return KINV_ERR_UNSUPPORTED;
  if (workspace_bytes < w.bytes) return KINV_ERR_WORKSPACE;
  TreeAttnParams p{};
  p.tree = *tree;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k_cache);
  p.v = static_cast<const __nv_bfloat16*>(v_cache);
  p.seq_stride = seq_stride;
  p.tok_stride = tok_stride;
  p.out = static_cast<__nv_bfloat16*>(out);
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
  p.ws_o = reinterpret_cast<float*>(ws + w.o);
  p.ws_ml = reinterpret_cast<float*>(ws + w.ml);
  p.ws_cov = reinterpret_cast<int*>(ws + w.cov);
  p.groups = static_cast<int>(w.groups);
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.gs = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
  p.S = static_cast<int>(S);
  p.c2 = base2_factor(scale, D);
  p.status = device_status_word();
  return D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}
