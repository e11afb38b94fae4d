// Attention over the 8-bit key/value cache, with or without a sliding window.
//
// A row's arithmetic is that of kinv_attn_decode on the cache read back (see
// attention.cu): 256-key splits at absolute offsets, the base-2 softmax, weights
// carried as a bf16 pair, one fp32 chain over 16-key steps, the left fold over
// the splits.  The codes enter the tensor cores exactly: a key's as f16 numbers, with q
// as f16 times a power of two of the row and head; a value's as the bf16 numbers that
// expand4() makes of them.  The powers of two that are missing are applied
// where they cost least, which is exact: a score is multiplied by its key's 2^E, and
// both halves of a weight by its value's 2^(E - Emax) (Emax the split's largest) and a
// constant, with the rest put back into the partial.  So the bits are those of attention
// over the cache read back wherever no score, product or sum on the way leaves fp32's
// normal range.
#include <math.h>

#include <cmath>

#include "attn_mma.cuh"
#include "attn_tc.cuh"
#include "cache8.cuh"
#include "cache8_read.cuh"
#include "common.cuh"
#include "window.cuh"

namespace kinv {
namespace {

constexpr int kSplit = kSplitKeys;
constexpr int kThreads = 256;  // eight warps, 32 keys each for the scores
constexpr int kPairs = 8;      // query heads per kv head, at most

struct Attn8Params {
  const __nv_bfloat16* q;
  Cache8View cache;
  const int32_t* kv_len;
  float* ws_o;   // [B][Hq][S][D]
  float* ws_ml;  // [B][Hq][S][2]
  int Hq, G, S, B;
  float c2;      // fp32(scale * log2 e)
  Window win;
  int* status;
  __nv_bfloat16* out;  // of the one-launch form
};

constexpr int kBox = 64;  // keys of one TMA copy

// D = A . B + D, one 16 x 8 x 16 warp MMA, f16 inputs, fp32 accumulation.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Blocks of a launch stay (three to an SM for D = 128, five for D = 64) and walk
// the listed splits of all sequences: block (g, p) takes kv head g of places p,
// p + gridDim.y, ... in the batch's one list of splits.  Each block has one K and
// one V buffer; the next split's K is requested when this one's scores are done,
// its V when this one's products are, so copies are in flight throughout.
//
// S^T = K . q^T and O^T = V^T . P^T: the codes are the A operand (16 keys x 16
// values, 16 values x 16 keys), so each is expanded once whatever the number of
// query heads, and the eight columns are the pairs.  Within a 16-value step of
// q . k the values are taken in another order on both sides (a lane's word holds
// four neighbours), which a step's sum does not depend on.
// GP = 4: at most four query heads per kv head; the lanes of the other four
// columns take half of the keys' softmax.
//
// ONE: a cluster per (sequence, kv head) with a block for each split that there can
// be, at most eight; the partials stay in shared memory and the cluster's blocks fold
// them together, so the call is one launch.
template <int D, bool I8, int GP, bool ONE>
__global__ void __launch_bounds__(kThreads, D == 128 ? 3 : 5)
    attn8_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const Attn8Params p) {
  constexpr int C = D / 16;           // 16-byte chunks of a key's codes
  constexpr int TILE = kSplit * D;    // bytes of a split's K or V codes
  constexpr int kLift = I8 ? 106 : 127;  // weights go in times 2^kLift: 256 products of 127 * 2^-6 or 448 * 2^-120 stay below 2^127
  constexpr int QROW = D * 2 + 16;    // bytes of a row of q (padded: eight rows in eight bank groups)
  constexpr int PHALF = GP * kSplit * 2;
  extern __shared__ __align__(1024) unsigned char smem[];
  // K, V; P hi and lo [GP][256] (before them, in the same place, q [8]); the factors; the warps' results
  unsigned char* pt = smem + 2 * TILE;
  constexpr int PQ = 2 * PHALF > 8 * QROW ? 2 * PHALF : 8 * QROW;
  float* fk = reinterpret_cast<float*>(pt + PQ);                          // [256] factors of the scores
  __nv_bfloat16* fv = reinterpret_cast<__nv_bfloat16*>(fk + kSplit);      // [256] factors of the weights
  float* wmax = reinterpret_cast<float*>(fv + kSplit);                    // [8 pairs][8 warps]
  float* wsum = wmax + 8 * kPairs;
  int* wexp = reinterpret_cast<int*>(wsum + 8 * kPairs);                  // [8]
  float* qc2 = reinterpret_cast<float*>(wexp + 8);                        // [8] the pairs' softmax factors
  uint64_t* bars = reinterpret_cast<uint64_t*>(qc2 + 8);                  // K, V
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t k_base = smem_addr(smem), v_base = k_base + TILE, pt_base = smem_addr(pt);
  const uint32_t k_bar = smem_addr(bars), v_bar = smem_addr(bars + 1);
  if (k_base & 1023u) {  // the copies' swizzle goes by address bits
    if (t == 0 && p.status) atomicExch(p.status, DEV_TIMEOUT_ATTN);
    return;
  }
  if (t == 0) {
    mbar_init(k_bar, 1);
    mbar_init(v_bar, 1);
    fence_mbar_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();

  // The walk: lane j holds the length of sequence wb + j and the number of listed
  // splits of sequences wb .. wb + j; `base` splits lie before wb.
  const int g = ONE ? blockIdx.x / p.S : blockIdx.x, G = p.G;
  int wb = 0, base = 0, wlen = 0, winc = 0;
  auto load_window = [&]() {
    const int b = wb + lane;
    wlen = b < p.B ? p.kv_len[b] : 0;
    if (wlen < 0 || wlen > p.cache.slots) wlen = 0;  // the merge kernel reports it
    winc = wlen > 0 ? visible_splits(p.win, window_lo(p.win, wlen), wlen).count : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += x;
    }
  };
  struct Item {
    int b, i, k0, cnt, lo, sink;  // b < 0: none
  };
  auto visible = [](const Item& x, int key) { return key < x.cnt && (key >= x.lo || key < x.sink); };
  auto item_at = [&](int at) {
    Item x;
    x.b = -1;
    int total;
    while (at >= base + (total = __shfl_sync(0xffffffffu, winc, 31))) {
      base += total;
      wb += 32;
      if (wb >= p.B) return x;
      load_window();
    }
    const int rel = at - base;
    const int j = __popc(__ballot_sync(0xffffffffu, winc <= rel));
    const int before = j > 0 ? __shfl_sync(0xffffffffu, winc, j - 1) : 0;
    const int len = __shfl_sync(0xffffffffu, wlen, j);
    const int first = window_lo(p.win, len);
    x.b = wb + j;
    x.i = rel - before;
    x.k0 = visible_splits(p.win, first, len).split(x.i) * kSplit;
    x.cnt = min(kSplit, len - x.k0);
    x.lo = first - x.k0;
    x.sink = p.win.sinks - x.k0;
    return x;
  };
  const uint64_t policy = l2_policy_evict_first();  // each code is read once per step
  auto request = [&](const CUtensorMap* map, const Item& x, uint32_t dst, uint32_t bar) {
    uint32_t live = 0;
#pragma unroll
    for (int j = 0; j < kSplit / kBox; ++j)
      if (j * kBox < x.cnt && (j * kBox < x.sink || (j + 1) * kBox > x.lo)) live |= 1u << j;
    mbar_arrive_expect_tx(bar, __popc(live) * kBox * D);
#pragma unroll
    for (int j = 0; j < kSplit / kBox; ++j)
      if (live >> j & 1) tma_load_4d(dst + j * kBox * D, map, 0, g, x.k0 + j * kBox, x.b, bar, policy);
  };
  // what a thread holds of the next split: its key's exponents, and four values (D = 64: lanes 0-15) of query head `warp`
  int ek, ev;
  uint2 qv;
  auto fetch = [&](const Item& x) {
    ek = ev = kExpNaN;
    if (visible(x, t)) {
      const int64_t e = x.b * p.cache.eseq_stride + g * p.cache.ehead_stride + x.k0 + t;
      ek = p.cache.ke[e];
      ev = p.cache.ve[e];
    }
    qv = make_uint2(0, 0);
    if (warp < G && lane < D / 4)
      qv = *reinterpret_cast<const uint2*>(p.q + (static_cast<int64_t>(x.b) * p.Hq + g * G + warp) * D + 4 * lane);
  };
  // chunk c of row r of a buffer (the copies' swizzle): the eight rows of an
  // ldmatrix phase fall in eight different bank groups
  auto at = [](int r, int c) {
    return static_cast<uint32_t>(r * D + ((C == 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
  };

  int place = blockIdx.y, one_len = 0, one_count = 0;
  Item cur;
  if (ONE) {
    one_len = p.kv_len[blockIdx.y];
    const int rank = blockIdx.x - g * p.S;
    if (one_len < 0 || one_len > p.cache.slots) {
      if (t == 0 && p.status) atomicExch(p.status, DEV_ATTN_BAD_LENGTH);
      one_len = 0;
    }
    const int first = window_lo(p.win, one_len);
    const SplitList list = visible_splits(p.win, first, one_len);
    one_count = list.count;
    cur.b = rank < one_count ? static_cast<int>(blockIdx.y) : -1;
    cur.i = rank;
    cur.k0 = list.split(rank) * kSplit;
    cur.cnt = min(kSplit, one_len - cur.k0);
    cur.lo = first - cur.k0;
    cur.sink = p.win.sinks - cur.k0;
  } else {
    load_window();
    cur = item_at(place);
    if (cur.b < 0) return;
  }
  float* one_o = reinterpret_cast<float*>(smem);  // over K, once the scores are done: [8 pairs][D], then (m, l) [8]
  if (cur.b >= 0 && t == 0) {
    request(&tmK, cur, k_base, k_bar);
    request(&tmV, cur, v_base, v_bar);
  }
  if (cur.b >= 0) fetch(cur);
  for (uint32_t phase = 0; cur.b >= 0; phase ^= 1) {
    // this split's factors and q into shared memory; the next one's requested
    const int my_ev = ev;
    const bool my_vis = visible(cur, t);
    fk[t] = exponent_factor(ek);
    {
      const int wm = __reduce_max_sync(0xffffffffu, my_ev);
      if (lane == 0) wexp[warp] = wm;
      // q of head `warp` as f16 times 2^up
      const uint32_t qm = __vmaxu2(qv.x & 0x7FFF7FFFu, qv.y & 0x7FFF7FFFu);
      const int top = static_cast<int>(__reduce_max_sync(0xffffffffu, max(qm & 0xFFFFu, qm >> 16)) >> 7);
      const int up = min(141 - min(top, 254), 120);
      const float f = exponent_factor(up);
      if (lane == 0) qc2[warp] = __fmul_rn(p.c2, exponent_factor(-up));
      if (lane < D / 4) {
        // of each sixteen values 0, 1, 4, 5, 8, ..., then the others
        const __half2 a = __floats2half2_rn(__fmul_rn(bf16_lo(qv.x), f), __fmul_rn(bf16_hi(qv.x), f));
        const __half2 c = __floats2half2_rn(__fmul_rn(bf16_lo(qv.y), f), __fmul_rn(bf16_hi(qv.y), f));
        unsigned char* to = pt + warp * QROW + (lane >> 2) * 32 + (lane & 3) * 4;
        *reinterpret_cast<__half2*>(to) = a;
        *reinterpret_cast<__half2*>(to + 16) = c;
      }
    }
    Item next;
    next.b = -1;
    if (!ONE) {
      place += gridDim.y;
      next = item_at(place);
      if (next.b >= 0) fetch(next);
    }
    bool ok = mbar_wait_bounded(k_bar, phase, p.status, DEV_TIMEOUT_ATTN);
    if (__syncthreads_or(!ok)) {
      mbar_wait_bounded(v_bar, phase, nullptr, 0);  // the copy in flight lands before the block leaves
      break;
    }
    const int4 e0 = *reinterpret_cast<const int4*>(wexp), e1 = *reinterpret_cast<const int4*>(wexp + 4);
    const int ev_max = max(max(max(e0.x, e0.y), max(e0.z, e0.w)), max(max(e1.x, e1.y), max(e1.z, e1.w)));
    // 0 for a hidden key, whose weight is 0
    const int fe = !my_vis ? 0 : my_ev == kExpNaN ? 0x7FFF : max(my_ev - ev_max + 127 + kLift, 0) << 7;
    fv[t] = __ushort_as_bfloat16(static_cast<unsigned short>(fe));

    // --- scores: warp w owns keys 32w .. 32w + 31, two 16-key tiles
    float sc[2][4] = {};
    // the 32-key groups that hold a visible key: the others add nothing
    const bool whole = cur.cnt == kSplit && (cur.lo <= 0 || cur.sink >= kSplit);  // no key hidden: no mask
    uint32_t groups = 0xFF;
    if (!whole) {
      groups = 0;
#pragma unroll
      for (int j = 0; j < kSplit / 32; ++j)
        if (j * 32 < cur.cnt && (j * 32 < cur.sink || (j + 1) * 32 > cur.lo)) groups |= 1u << j;
    }
    if (groups >> warp & 1) {
      uint32_t qb[C][2];  // q fragments (B operand: 16 values x 8 pairs)
#pragma unroll
      for (int kp = 0; kp < C / 2; ++kp)
        ldsm_x4(pt_base + (lane & 7) * QROW + kp * 64 + (lane >> 3) * 16, qb[2 * kp][0], qb[2 * kp][1],
                qb[2 * kp + 1][0], qb[2 * kp + 1][1]);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int row = warp * 32 + mt * 16 + (lane & 15);
#pragma unroll
        for (int kp = 0; kp < C / 2; ++kp) {
          // matrices: rows 0-7 and 8-15 of chunk 2kp, then of chunk 2kp + 1
          uint32_t w0, w1, w2, w3, a[4];
          ldsm_x4(k_base + at(row, 2 * kp + (lane >> 4)), w0, w1, w2, w3);
          expand4_f16<I8>(w0, a[0], a[2]);
          expand4_f16<I8>(w1, a[1], a[3]);
          mma_f16_16816(sc[mt], a, qb[2 * kp][0], qb[2 * kp][1]);
          expand4_f16<I8>(w2, a[0], a[2]);
          expand4_f16<I8>(w3, a[1], a[3]);
          mma_f16_16816(sc[mt], a, qb[2 * kp + 1][0], qb[2 * kp + 1][1]);
        }
        // rows gq and gq + 8 of the tile: columns (pairs) 2tq, 2tq + 1
        const float f0 = fk[warp * 32 + mt * 16 + gq], f1 = fk[warp * 32 + mt * 16 + 8 + gq];
        sc[mt][0] = __fmul_rn(sc[mt][0], f0);
        sc[mt][1] = __fmul_rn(sc[mt][1], f0);
        sc[mt][2] = __fmul_rn(sc[mt][2], f1);
        sc[mt][3] = __fmul_rn(sc[mt][3], f1);
      }
    }
    // Lanes gq and gq ^ 1 swap, so that a lane holds keys 8nb + 2 kq + e (kq =
    // gq / 2) of one pair, 2tq + (gq & 1): the layout that the sums are ordered by.
    const int kq = gq >> 1;
    float y[4][2];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const float mine0 = sc[nb >> 1][2 * (nb & 1)], mine1 = sc[nb >> 1][2 * (nb & 1) + 1];
      const float got = __shfl_xor_sync(0xffffffffu, (gq & 1) ? mine0 : mine1, 4);
      y[nb][0] = (gq & 1) ? got : mine0;
      y[nb][1] = (gq & 1) ? mine1 : got;
    }
    // GP = 4: lanes tq >= 2 (pairs 4 .. 7, which are none) take blocks nb = 2, 3 of lane tq - 2
    constexpr int NB = GP == 4 ? 2 : 4;
    const int nb0 = GP == 4 && tq >= 2 ? 2 : 0;
    const int pair = GP == 4 ? 2 * (tq & 1) + (gq & 1) : 2 * tq + (gq & 1);
    float x[NB][2];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[i][e] = y[i][e];
        if (GP == 4) {
          const float got = __shfl_xor_sync(0xffffffffu, y[2 + i][e], 2);
          if (tq >= 2) x[i][e] = got;
        }
      }
    const int key0 = warp * 32 + nb0 * 8 + 2 * kq;
    float mx = -INFINITY;
    if (whole) {
#pragma unroll
      for (int i = 0; i < NB; ++i) mx = fmax3(mx, x[i][0], x[i][1]);
    } else {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (visible(cur, key0 + 8 * i + e)) mx = fmaxf(mx, x[i][e]);
    }
#pragma unroll
    for (int o = GP == 4 ? 2 : 8; o <= 16; o = o == 2 ? 8 : o << 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (kq == 0) wmax[pair * 8 + warp] = mx;
    __syncthreads();
    if (t == 0 && next.b >= 0) request(&tmK, next, k_base, k_bar);  // every warp is done with K
    const float4 m0 = *reinterpret_cast<const float4*>(wmax + pair * 8), m1 = *reinterpret_cast<const float4*>(wmax + pair * 8 + 4);
    const float c2 = qc2[pair];
    const float m = __fmul_rn(fmaxf(fmax3(fmax3(m0.x, m0.y, m0.z), m0.w, m1.x), fmax3(m1.y, m1.z, m1.w)), c2);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) x[i][e] = ex2_approx(__fmaf_rn(x[i][e], c2, -m));
    if (!whole) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!visible(cur, key0 + 8 * i + e)) x[i][e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      // the weight's halves, then their factor (exact: a power of two)
      const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162*>(fv + key0 + 8 * i);
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[i][0], x[i][1]);
      const float2 hf = __bfloat1622float2(h);
      const __nv_bfloat162 l = __floats2bfloat162_rn(__fsub_rn(x[i][0], hf.x), __fsub_rn(x[i][1], hf.y));
      const uint32_t to = static_cast<uint32_t>(pair * kSplit * 2 + (((warp * 4 + nb0 + i) ^ pair) << 4) + 4 * kq);
      *reinterpret_cast<__nv_bfloat162*>(pt + to) = __hmul2(h, f);
      *reinterpret_cast<__nv_bfloat162*>(pt + PHALF + to) = __hmul2(l, f);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) sum = __fadd_rn(sum, x[i][e]);
    if (GP == 4) {  // the sum goes on from blocks 0, 1 to blocks 2, 3
      const float got = __shfl_xor_sync(0xffffffffu, sum, 2);
      sum = got;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) sum = __fadd_rn(sum, x[i][e]);
    }
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
    if (kq == 0 && (GP == 8 || tq >= 2)) wsum[warp * kPairs + pair] = sum;
    ok = mbar_wait_bounded(v_bar, phase, p.status, DEV_TIMEOUT_ATTN);
    if (__syncthreads_or(!ok)) {
      if (next.b >= 0) mbar_wait_bounded(k_bar, phase ^ 1, nullptr, 0);
      break;
    }

    // --- O^T = V^T . P^T: warp w owns values 16w .. 16w + 15 over all 256 keys,
    // one chain of sixteen 16-key steps, each its high halves, then its low ones
    if (warp < C) {
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      const int prow = lane & (GP - 1);  // GP = 4: columns 4 .. 7 repeat, and are not used
#pragma unroll 2
      for (int kk = 0; kk < kSplit / 32; ++kk) {
        if (!(groups >> kk & 1)) continue;
        // transposed 8 x 8 matrices of byte pairs: keys 8i .. 8i + 7 of the 32
        uint32_t w[4], bh[4], bl[4], a[4];
        ldsm_x4_t(v_base + at(kk * 32 + lane, warp), w[0], w[1], w[2], w[3]);
        const uint32_t from = static_cast<uint32_t>(prow * kSplit * 2 + (((4 * kk + (lane >> 3)) ^ prow) << 4));
        ldsm_x4(pt_base + from, bh[0], bh[1], bh[2], bh[3]);
        ldsm_x4(pt_base + PHALF + from, bl[0], bl[1], bl[2], bl[3]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          // rows gq: value 2gq, rows gq + 8: value 2gq + 1
          expand4<I8>(w[2 * s], a[0], a[1]);
          expand4<I8>(w[2 * s + 1], a[2], a[3]);
          mma_bf16_16816(o, a, bh[2 * s], bh[2 * s + 1]);
          mma_bf16_16816(o, a, bl[2 * s], bl[2 * s + 1]);
        }
      }
      // 2^Emax and the constants back, the smaller factor first (no intermediate
      // result is smaller than the product)
      const float back0 = exponent_factor(min(ev_max, 0)), back1 = exponent_factor(max(ev_max, 0) + expand_exp<I8>() - kLift);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __fmul_rn(__fmul_rn(o[i], back0), back1);
      const int64_t row = static_cast<int64_t>(cur.b) * p.Hq + g * G;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (ONE)
          *reinterpret_cast<float2*>(one_o + (2 * tq + e) * D + warp * 16 + 2 * gq) = make_float2(o[e], o[2 + e]);
        else if (2 * tq + e < G)
          *reinterpret_cast<float2*>(p.ws_o + ((row + 2 * tq + e) * p.S + cur.i) * D + warp * 16 + 2 * gq) =
              make_float2(o[e], o[2 + e]);
      if (warp == 0 && kq == 0 && pair < G && (GP == 8 || tq >= 2)) {
        float l = wsum[pair];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) l = __fadd_rn(l, wsum[w * kPairs + pair]);
        *reinterpret_cast<float2*>(ONE ? one_o + kPairs * D + 2 * pair : p.ws_ml + ((row + pair) * p.S + cur.i) * 2) =
            make_float2(m, l);
      }
    }
    if (next.b < 0) break;
    __syncthreads();  // every warp is done with V, P and the sums
    if (t == 0) request(&tmV, next, v_base, v_bar);
    cur = next;
  }
  if (ONE) {
    cluster_sync();
    fold_cluster<D, kThreads>(k_base, kPairs, G, blockIdx.x - g * p.S, p.S, one_count,
                              p.out + (static_cast<int64_t>(blockIdx.y) * p.Hq + g * G) * D);
    cluster_sync();  // no block leaves while its partial is read
  }
}

template <int D, int GP>
constexpr size_t split8_smem_bytes() {
  constexpr size_t P = 2 * static_cast<size_t>(GP) * kSplit * 2, Q = 8 * (D * 2 + 16);
  return 2 * static_cast<size_t>(kSplit) * D + (P > Q ? P : Q) + kSplit * 6 + 2 * 8 * kPairs * 4 + 2 * 8 * 4 + 2 * 8;
}

// The codes as bytes (D, Hkv, slots, B), boxes of 64 keys of one head, rows of
// 128 bytes in the 128-byte swizzle or of 64 in the 64-byte one.
inline bool encode_codes(CUtensorMap* map, const void* ptr, const Cache8View& c, int B, int Hkv, int D) {
  auto fn = tma_encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(c.slots),
                              static_cast<cuuint64_t>(B)};
  // one sequence: any sequence stride describes it (the coordinate is 0)
  const cuuint64_t seq = B > 1 ? c.seq_stride : static_cast<cuuint64_t>(c.slots) * c.tok_stride;
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(c.tok_stride), seq};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(D), 1, kBox, 1}, step[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool I8, int GP>
kinv_status launch_decode8(const Attn8Params& p, const MergeParams& mp, int Hkv, cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!encode_codes(&mk, p.cache.k, p.cache, p.B, Hkv, D) || !encode_codes(&mv, p.cache.v, p.cache, p.B, Hkv, D))
    return KINV_ERR_UNSUPPORTED;
  constexpr size_t smem = split8_smem_bytes<D, GP>();
  const int64_t resident = static_cast<int64_t>(sm_count()) * (D == 128 ? 3 : 5);
  const int64_t most = static_cast<int64_t>(p.B) * p.S;
  // One launch of clusters where there are at most eight splits a row and all blocks
  // run at once; clusters of more than four need more room to be placed (32/8 heads of
  // 128: one request of 500 keys 8.2 us against 10.2, 24 of 500 10.4 against 12.4, 3 of
  // 2,048 8.6 against 10.3, but 7 of 2,048, 448 blocks, 14.4 against 12.3).
  if (p.S <= 8 && most * Hkv <= (p.S <= 4 ? resident : 2 * resident / 3)) {
    auto one = attn8_split_kernel<D, I8, GP, true>;
    const kinv_status st = ensure_smem(reinterpret_cast<const void*>(one), smem);
    if (st != KINV_OK) return st;
    return launch_kernel(one, dim3(Hkv * p.S, p.B), dim3(kThreads), smem, stream, p.S, mk, mv, p);
  }
  auto kernel = attn8_split_kernel<D, I8, GP, false>;
  kinv_status st = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
  if (st != KINV_OK) return st;
  // as many blocks as the GPU holds at a time, or as there can be splits
  int64_t places = (resident + Hkv - 1) / Hkv;
  if (places > most) places = most;
  st = launch_kernel(kernel, dim3(Hkv, static_cast<unsigned>(places)), dim3(kThreads), smem, stream, 1, mk, mv, p);
  if (st != KINV_OK) return st;
  return launch_window_merge<D>(mp, p.B, stream);
}

template <int D, bool I8>
kinv_status launch_decode8(const Attn8Params& p, const MergeParams& mp, int Hkv, cudaStream_t stream) {
  if (p.S == 0) return launch_window_merge<D>(mp, p.B, stream);
  return p.G <= 4 ? launch_decode8<D, I8, 4>(p, mp, Hkv, stream) : launch_decode8<D, I8, 8>(p, mp, Hkv, stream);
}

size_t decode8_bytes(int64_t B, int Hq, int D, int64_t S) {
  const size_t o = static_cast<size_t>(B) * Hq * S * D * 4;
  return (o + 255) / 256 * 256 + static_cast<size_t>(B) * Hq * S * 8;
}

kinv_status check_heads(int Hq, int Hkv, int split_len, int window, int sinks) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || window < 0 || sinks < 0) return KINV_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if ((G != 1 && G != 2 && G != 4 && G != kPairs) || split_len != kSplit) return KINV_ERR_UNSUPPORTED;
  return KINV_OK;
}

}  // namespace
}  // namespace kinv

using namespace kinv;

extern "C" size_t kinv_attn_decode8_workspace(int B, int Hq, int D, int slots, int window, int sinks, int split_len) {
  if (B <= 0 || Hq <= 0 || D <= 0 || slots <= 0 || window < 0 || sinks < 0 || split_len != kSplit) return 0;
  return decode8_bytes(B, Hq, D, max_visible_splits(window, sinks, slots));
}

extern "C" kinv_status kinv_attn_decode8(const void* q, const kinv_cache8* cache, const int32_t* kv_len, void* out,
                                         int B, int Hq, int Hkv, int D, int split_len, int window, int sinks,
                                         float scale, void* workspace, size_t ws_bytes, kinv_stream stream) {
  if (B < 0) return KINV_ERR_INVALID_ARG;
  Attn8Params p{};
  kinv_status st = check_heads(Hq, Hkv, split_len, window, sinks);
  if (st == KINV_OK) st = check_cache8(cache, Hkv, D, &p.cache);
  if (st != KINV_OK) return st;
  if (B > cache->B) return KINV_ERR_INVALID_ARG;
  if (B == 0) return KINV_OK;
  if (!q || !out || !kv_len || (!workspace && cache->slots > 0)) return KINV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return KINV_ERR_ALIGNMENT;
  const int64_t S = max_visible_splits(window, sinks, cache->slots);  // 0 for a cache of no slots
  const bool i8 = cache->dtype == KINV_I8;
  p.c2 = base2_factor(scale, D);
  if (B > 1 && cache->seq_stride == 0) return KINV_ERR_INVALID_ARG;
  if (B > 65535 || B * S > 0x7F000000) return KINV_ERR_UNSUPPORTED;
  if (ws_bytes < decode8_bytes(B, Hq, D, S)) return KINV_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv_len = kv_len;
  p.ws_o = static_cast<float*>(workspace);
  const size_t o_bytes = static_cast<size_t>(B) * Hq * S * D * 4;
  p.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + (o_bytes + 255) / 256 * 256);
  p.Hq = Hq;
  p.G = Hq / Hkv;
  p.S = static_cast<int>(S);
  p.B = B;
  p.win = Window{window, sinks};
  p.status = device_status_word();
  p.out = static_cast<__nv_bfloat16*>(out);
  MergeParams mp{p.ws_o, p.ws_ml, kv_len, static_cast<__nv_bfloat16*>(out), Hq, p.S, cache->slots, p.win, p.status};
  if (D == 128)
    return i8 ? launch_decode8<128, true>(p, mp, Hkv, stream) : launch_decode8<128, false>(p, mp, Hkv, stream);
  return i8 ? launch_decode8<64, true>(p, mp, Hkv, stream) : launch_decode8<64, false>(p, mp, Hkv, stream);
}

namespace kinv {
namespace {
size_t read_back_bytes(int B, int max_kv, int Hkv, int D) { return static_cast<size_t>(B) * max_kv * Hkv * D * 4; }
}  // namespace
}  // namespace kinv

// A prompt chunk: the keys and values that its rows see, read back into the
// workspace, then kinv_attn_prefill's kernel.
extern "C" size_t kinv_attn_prefill8_workspace(int B, int total_rows, int Hq, int Hkv, int D, int max_kv,
                                               int split_len) {
  if (B <= 0 || total_rows <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_kv <= 0 || split_len != kSplit) return 0;
  return read_back_bytes(B, max_kv, Hkv, D) + most_parts_bytes(B, total_rows, Hq, Hkv, D, max_kv);
}

extern "C" kinv_status kinv_attn_prefill8(const void* q, const kinv_cache8* cache, const int32_t* q_start,
                                          const int32_t* q_len, const int32_t* q_offset, void* out, int B,
                                          int total_rows, int max_q_len, int max_kv, int Hq, int Hkv, int D,
                                          int split_len, int window, int sinks, float scale, void* workspace,
                                          size_t ws_bytes, kinv_stream stream) {
  if (B < 0 || total_rows < 0 || max_q_len < 0 || max_kv < 0) return KINV_ERR_INVALID_ARG;
  ReadParams r{};
  kinv_status st = check_heads(Hq, Hkv, split_len, window, sinks);
  if (st == KINV_OK) st = check_cache8(cache, Hkv, D, &r.cache);
  if (st != KINV_OK) return st;
  if (B > cache->B || max_kv > cache->slots) return KINV_ERR_INVALID_ARG;
  if (B == 0 || total_rows == 0 || max_q_len == 0) return KINV_OK;
  if (!q || !out || !q_start || !q_len || !q_offset || !workspace || max_kv <= 0) return KINV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return KINV_ERR_ALIGNMENT;
  const int tile_rows = 128 / (Hq / Hkv);  // of the prefill kernel, which counts its tiles in an int
  if (B > 65535 || (static_cast<int64_t>(max_q_len) + tile_rows - 1) / tile_rows * Hkv * B > 0x7F000000)
    return KINV_ERR_UNSUPPORTED;
  const size_t need = read_back_bytes(B, max_kv, Hkv, D);
  if (ws_bytes < need) return KINV_ERR_WORKSPACE;
  r.k = static_cast<__nv_bfloat16*>(workspace);
  r.v = r.k + need / 4;
  r.tok_stride = static_cast<int64_t>(Hkv) * D;
  r.seq_stride = r.tok_stride * max_kv;
  r.q_start = q_start;
  r.q_len = q_len;
  r.max_len = max_kv;
  r.max_q_len = max_q_len;
  r.Hkv = Hkv;
  r.win = Window{window, sinks};
  r.status = nullptr;
  st = launch_cache8_read(r, cache->dtype == KINV_I8, B, D, stream);
  if (st != KINV_OK) return st;
  return kinv_attn_prefill_window(q, r.k, r.v, r.seq_stride, r.tok_stride, q_start, q_len, q_offset, out, B,
                                  total_rows, max_q_len, max_kv, Hq, Hkv, D, split_len, window, sinks, scale,
                                  static_cast<char*>(workspace) + need, ws_bytes - need, stream);
}
