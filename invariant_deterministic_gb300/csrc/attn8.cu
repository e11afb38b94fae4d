// Attention over the 8-bit key/value cache, with or without a sliding window.
//
// A row's arithmetic is that of kinv_attn_decode on the cache read back (see
// attention.cu): 256-key splits at absolute offsets, the base-2 softmax, weights
// carried as a bf16 pair, one fp32 chain over 16-key steps, the left fold over
// the splits.  The codes enter the tensor cores as the bf16 numbers that
// expand4() makes of them, and the powers of two that are missing are applied
// where they cost least, which is exact: q is multiplied by 2^90 for e4m3 (whose
// codes stand there times 2^-120), a score by its key's 2^E, and both halves of a
// weight by its value's 2^(E - Emax) (Emax the split's largest) and a constant,
// with the rest put back into the partial.  So the bits are those of attention over the
// cache read back wherever no score, product or sum on the way leaves fp32's
// normal range.
#include <math.h>

#include <cmath>

#include "attn_mma.cuh"
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
  int Hq, G, S;
  float c2;      // fp32(scale * log2 e), times 2^30 for e4m3
  Window win;
  int* status;
};

// One block per (kv head, listed split, sequence).  S^T = K . q^T and
// O^T = V^T . P^T: the codes are the A operand (16 keys x 16 values, 16 values x
// 16 keys), so each is expanded once whatever the number of query heads, and the
// eight columns are the pairs.  Within a 16-value step of q . k the values are
// taken in another order on both sides (0, 2, 4, 6, ... as the bytes of a word
// come apart), which a step's sum does not depend on.
template <int D, bool I8>
__global__ void __launch_bounds__(kThreads) attn8_split_kernel(const Attn8Params p) {
  constexpr int C = D / 16;           // 16-byte chunks of a key's codes
  constexpr int TILE = kSplit * D;    // bytes of a split's K or V codes
  constexpr int kLift = I8 ? 100 : 127;  // weights go in times 2^kLift: 256 products of 127 or 448 * 2^-120 stay below 2^127
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* pt = smem + 2 * TILE;             // P hi [8][256] bf16, then lo
  float* fk = reinterpret_cast<float*>(pt + 2 * kPairs * kSplit * 2);    // [256] factors of the scores
  __nv_bfloat16* fv = reinterpret_cast<__nv_bfloat16*>(fk + kSplit);      // [256] factors of the weights
  __shared__ float wmax[kThreads / 32][kPairs], wsum[kThreads / 32][kPairs];
  __shared__ int wexp[kThreads / 32];

  pdl_launch_dependents();
  pdl_wait();
  const int g = blockIdx.x, b = blockIdx.z;
  const int len = p.kv_len[b];
  if (len <= 0 || len > p.cache.slots) return;  // the merge kernel reports a length out of bounds
  const int lo_key = window_lo(p.win, len);
  const SplitList list = visible_splits(p.win, lo_key, len);
  if (static_cast<int>(blockIdx.y) >= list.count) return;
  const int k0 = list.split(blockIdx.y) * kSplit;
  const int cnt = min(kSplit, len - k0);       // keys of the split
  const int lo = lo_key - k0, sink = p.win.sinks - k0;
  auto visible = [&](int key) { return key < cnt && (key >= lo || key < sink); };
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int G = p.G;
  const uint32_t k_base = smem_addr(smem), v_base = k_base + TILE, pt_base = smem_addr(pt);

  // chunk c of row r sits at chunk slot(r, c): the eight rows of an ldmatrix
  // phase fall in eight different bank groups
  auto at = [](int r, int c) {
    return static_cast<uint32_t>(r * D + ((C == 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
  };
  const uint64_t policy = l2_policy_evict_first();
  const int64_t off = b * p.cache.seq_stride + static_cast<int64_t>(k0) * p.cache.tok_stride + g * D;
  auto load = [&](const unsigned char* src, uint32_t dst) {
#pragma unroll
    for (int it = 0; it < kSplit * C / kThreads; ++it) {
      const int idx = it * kThreads + t;
      const int r = idx / C, c = idx % C;
      if (visible(r)) cp_async16_hint(dst + at(r, c), src + off + static_cast<int64_t>(r) * p.cache.tok_stride + c * 16, policy);
    }
    cp_async_commit();
  };
  load(p.cache.k, k_base);
  load(p.cache.v, v_base);

  // this thread's key: its exponents
  int ek = kExpNaN, ev = kExpNaN;
  {
    const int64_t e = b * p.cache.eseq_stride + g * p.cache.ehead_stride + k0 + t;
    if (visible(t)) {
      ek = p.cache.ke[e];
      ev = p.cache.ve[e];
    }
  }
  // q fragments (B operand: 16 values x 8 pairs): lane (gq, tq) holds values
  // 4tq .. 4tq + 3 of each step, as (0, 2) and (1, 3)
  uint32_t qb[C][2];
  {
    const __nv_bfloat16* q = p.q + (static_cast<int64_t>(b) * p.Hq + g * G + gq) * D + 4 * tq;
#pragma unroll
    for (int ks = 0; ks < C; ++ks) {
      uint2 x = make_uint2(0, 0);
      if (gq < G) x = *reinterpret_cast<const uint2*>(q + 16 * ks);
      if (!I8) {
        const __nv_bfloat162 lift = __float2bfloat162_rn(0x1p90f);
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&x);
        h[0] = __hmul2(h[0], lift);
        h[1] = __hmul2(h[1], lift);
      }
      qb[ks][0] = __byte_perm(x.x, x.y, 0x5410);
      qb[ks][1] = __byte_perm(x.x, x.y, 0x7632);
    }
  }
  fk[t] = exponent_factor(ek);
  const int wm = __reduce_max_sync(0xffffffffu, ev);
  if (lane == 0) wexp[warp] = wm;
  cp_async_wait<1>();
  __syncthreads();
  int ev_max = wexp[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) ev_max = max(ev_max, wexp[w]);
  // 0 for a hidden key, whose weight is 0
  const int fe = !visible(t) ? 0 : ev == kExpNaN ? 0x7FFF : max(ev - ev_max + 127 + kLift, 0) << 7;
  fv[t] = __ushort_as_bfloat16(static_cast<unsigned short>(fe));

  // --- scores: warp w owns keys 32w .. 32w + 31, two 16-key tiles
  float sc[2][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[mt][i] = 0.f;
    const int row = warp * 32 + mt * 16 + (lane & 15);
#pragma unroll
    for (int kp = 0; kp < C / 2; ++kp) {
      // matrices: rows 0-7 and 8-15 of chunk 2kp, then of chunk 2kp + 1
      uint32_t w0, w1, w2, w3, a[4];
      ldsm_x4(k_base + at(row, 2 * kp + (lane >> 4)), w0, w1, w2, w3);
      expand4<I8>(w0, a[0], a[2]);
      expand4<I8>(w1, a[1], a[3]);
      mma_bf16_16816(sc[mt], a, qb[2 * kp][0], qb[2 * kp][1]);
      expand4<I8>(w2, a[0], a[2]);
      expand4<I8>(w3, a[1], a[3]);
      mma_bf16_16816(sc[mt], a, qb[2 * kp + 1][0], qb[2 * kp + 1][1]);
    }
    // rows gq and gq + 8 of the tile: columns (pairs) 2tq, 2tq + 1
    const float f0 = fk[warp * 32 + mt * 16 + gq], f1 = fk[warp * 32 + mt * 16 + 8 + gq];
    sc[mt][0] = __fmul_rn(sc[mt][0], f0);
    sc[mt][1] = __fmul_rn(sc[mt][1], f0);
    sc[mt][2] = __fmul_rn(sc[mt][2], f1);
    sc[mt][3] = __fmul_rn(sc[mt][3], f1);
  }
  // Lanes gq and gq ^ 1 swap, so that a lane holds keys 8nb + 2 kq + e (kq =
  // gq / 2) of one pair, 2tq + (gq & 1): the layout that the sums are ordered by.
  const int kq = gq >> 1, pair = 2 * tq + (gq & 1);
  float x[4][2];
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
    const float mine0 = sc[nb >> 1][2 * (nb & 1)], mine1 = sc[nb >> 1][2 * (nb & 1) + 1];
    const float got = __shfl_xor_sync(0xffffffffu, (gq & 1) ? mine0 : mine1, 4);
    x[nb][0] = (gq & 1) ? got : mine0;
    x[nb][1] = (gq & 1) ? mine1 : got;
  }
  bool see[4][2];
  float mx = -INFINITY;
#pragma unroll
  for (int nb = 0; nb < 4; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      see[nb][e] = visible(warp * 32 + nb * 8 + 2 * kq + e);
      if (see[nb][e]) mx = fmaxf(mx, x[nb][e]);
    }
#pragma unroll
  for (int o = 8; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (kq == 0) wmax[warp][pair] = mx;
  __syncthreads();
  float m = wmax[0][pair];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, wmax[w][pair]);
  m = __fmul_rn(m, p.c2);
  float sum = 0.f;
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
    const int key = warp * 32 + nb * 8 + 2 * kq;
    // the weight's halves, then their factor (exact: a power of two)
    const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162*>(fv + key);
    float w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      w[e] = see[nb][e] ? ex2_approx(__fmaf_rn(x[nb][e], p.c2, -m)) : 0.f;
      sum = __fadd_rn(sum, w[e]);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(w[0], w[1]);
    const float2 hf = __bfloat1622float2(h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(__fsub_rn(w[0], hf.x), __fsub_rn(w[1], hf.y));
    const uint32_t to = static_cast<uint32_t>(pair * kSplit * 2 + (((warp * 4 + nb) ^ pair) << 4) + 4 * kq);
    *reinterpret_cast<__nv_bfloat162*>(pt + to) = __hmul2(h, f);
    *reinterpret_cast<__nv_bfloat162*>(pt + kPairs * kSplit * 2 + to) = __hmul2(l, f);
  }
#pragma unroll
  for (int o = 8; o <= 16; o <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
  if (kq == 0) wsum[warp][pair] = sum;
  cp_async_wait<0>();
  __syncthreads();

  // --- O^T = V^T . P^T: warp w owns values 16w .. 16w + 15 over all 256 keys,
  // one chain of sixteen 16-key steps, each its high halves, then its low ones
  if (warp < C) {
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int kk = 0; kk < kSplit / 32; ++kk) {
      // transposed 8 x 8 matrices of byte pairs: keys 8i .. 8i + 7 of the 32
      uint32_t w[4], bh[4], bl[4], a[4];
      ldsm_x4_t(v_base + at(kk * 32 + lane, warp), w[0], w[1], w[2], w[3]);
      const uint32_t from = static_cast<uint32_t>((lane & 7) * kSplit * 2 + (((4 * kk + (lane >> 3)) ^ (lane & 7)) << 4));
      ldsm_x4(pt_base + from, bh[0], bh[1], bh[2], bh[3]);
      ldsm_x4(pt_base + kPairs * kSplit * 2 + from, bl[0], bl[1], bl[2], bl[3]);
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
    const float back0 = exponent_factor(min(ev_max, 0)), back1 = exponent_factor(max(ev_max, 0) + (I8 ? 0 : 120) - kLift);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __fmul_rn(__fmul_rn(o[i], back0), back1);
    const int64_t row = static_cast<int64_t>(b) * p.Hq + g * G;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (2 * tq + e < G)
        *reinterpret_cast<float2*>(p.ws_o + ((row + 2 * tq + e) * p.S + blockIdx.y) * D + warp * 16 + 2 * gq) =
            make_float2(o[e], o[2 + e]);
    if (warp == 0 && kq == 0 && pair < G) {
      float l = wsum[0][pair];
#pragma unroll
      for (int w = 1; w < kThreads / 32; ++w) l = __fadd_rn(l, wsum[w][pair]);
      *reinterpret_cast<float2*>(p.ws_ml + ((row + pair) * p.S + blockIdx.y) * 2) = make_float2(m, l);
    }
  }
}

template <int D>
constexpr size_t split8_smem_bytes() {
  return 2 * static_cast<size_t>(kSplit) * D + 2 * static_cast<size_t>(kPairs) * kSplit * 2 + kSplit * 6;
}

template <int D, bool I8>
kinv_status launch_decode8(const Attn8Params& p, const MergeParams& mp, int Hkv, int B, cudaStream_t stream) {
  void (*kernel)(const Attn8Params) = attn8_split_kernel<D, I8>;
  constexpr size_t smem = split8_smem_bytes<D>();
  kinv_status st = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
  if (st != KINV_OK) return st;
  st = launch_kernel(kernel, dim3(Hkv, p.S, B), dim3(kThreads), smem, stream, 1, p);
  if (st != KINV_OK) return st;
  return launch_kernel(window_merge_kernel<D>, dim3(p.Hq, B), dim3(D), 0, stream, 1, mp);
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
  if (!q || !out || !kv_len || !workspace) return KINV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return KINV_ERR_ALIGNMENT;
  const int64_t S = cache->slots > 0 ? max_visible_splits(window, sinks, cache->slots) : 1;
  const bool i8 = cache->dtype == KINV_I8;
  p.c2 = base2_factor(scale, D) * (i8 ? 1.f : 0x1p30f);
  if (B > 65535 || S > 65535 || !std::isfinite(p.c2)) return KINV_ERR_UNSUPPORTED;
  if (ws_bytes < decode8_bytes(B, Hq, D, S)) return KINV_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv_len = kv_len;
  p.ws_o = static_cast<float*>(workspace);
  const size_t o_bytes = static_cast<size_t>(B) * Hq * S * D * 4;
  p.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + (o_bytes + 255) / 256 * 256);
  p.Hq = Hq;
  p.G = Hq / Hkv;
  p.S = static_cast<int>(S);
  p.win = Window{window, sinks};
  p.status = device_status_word();
  MergeParams mp{p.ws_o, p.ws_ml, kv_len, static_cast<__nv_bfloat16*>(out), Hq, p.S, cache->slots, p.win, p.status};
  if (D == 128)
    return i8 ? launch_decode8<128, true>(p, mp, Hkv, B, stream) : launch_decode8<128, false>(p, mp, Hkv, B, stream);
  return i8 ? launch_decode8<64, true>(p, mp, Hkv, B, stream) : launch_decode8<64, false>(p, mp, Hkv, B, stream);
}

// A prompt chunk: the keys and values that its rows see, read back into the
// workspace, then kinv_attn_prefill's kernel.
extern "C" size_t kinv_attn_prefill8_workspace(int B, int total_rows, int Hq, int Hkv, int D, int max_kv,
                                               int split_len) {
  if (B <= 0 || total_rows <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_kv <= 0 || split_len != kSplit) return 0;
  return static_cast<size_t>(B) * max_kv * Hkv * D * 4;
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
  const int tile_rows = 128 / (Hq / Hkv);  // of the prefill kernel
  if (B > 65535 || (static_cast<int64_t>(max_q_len) + tile_rows - 1) / tile_rows > 65535) return KINV_ERR_UNSUPPORTED;
  const size_t need = kinv_attn_prefill8_workspace(B, total_rows, Hq, Hkv, D, max_kv, split_len);
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
                                  total_rows, max_q_len, max_kv, Hq, Hkv, D, split_len, window, sinks, scale, nullptr,
                                  0, stream);
}
