// Attention over a sliding window with sinks: which keys a row sees, and which
// 256-key splits hold them.
//
// A row with `len` keys up to its own (its position is len - 1) sees key j < len
// if j >= len - window or j < sinks; window 0 means every key.  The splits stay
// at the absolute offsets 0, 256, 512, ... of attention without a window, so a
// row's sums keep one order whatever the batch or the chunking; splits without a
// visible key are left out, and hidden keys in the others have weight 0.
#pragma once

#include "common.cuh"

namespace kinv {

constexpr int kSplitKeys = 256;

struct Window {
  int window;  // 0: none
  int sinks;
};

// The splits that hold a key of [0, min(sinks, lo)) or of [lo, end), in order:
// 0 .. a - 1, then w0 .. ns - 1.  `lo` is the first key of the window (of the
// earliest row, for a tile of rows), `end` the last row's length.
struct SplitList {
  int a, w0, count;
  __host__ __device__ int split(int i) const { return i < a ? i : w0 + i - a; }
};

__host__ __device__ inline int window_lo(const Window& w, int len) {
  return w.window > 0 && len > w.window ? len - w.window : 0;
}

__host__ __device__ inline SplitList visible_splits(const Window& w, int lo, int end) {
  SplitList s;
  const int ns = (end + kSplitKeys - 1) / kSplitKeys;
  const int sink = w.sinks < lo ? w.sinks : lo;
  s.a = (sink + kSplitKeys - 1) / kSplitKeys;
  s.w0 = lo / kSplitKeys > s.a ? lo / kSplitKeys : s.a;
  s.count = s.a + ns - s.w0;
  return s;
}

// Most splits that a row of at most max_len keys can have in its list.
inline int64_t max_visible_splits(int window, int sinks, int max_len) {
  const int64_t all = (static_cast<int64_t>(max_len) + kSplitKeys - 1) / kSplitKeys;
  if (window <= 0) return all;
  const int64_t some = (static_cast<int64_t>(sinks) + kSplitKeys - 1) / kSplitKeys +
                       (static_cast<int64_t>(window) + kSplitKeys - 2) / kSplitKeys + 1;
  return some < all ? some : all;
}

// Bytes of the partials that kinv_attn_prefill_window may use for a call of at most
// most_rows rows of a sequence, whatever the window.
size_t most_parts_bytes(int B, int most_rows, int Hq, int Hkv, int D, int max_kv);

// The fold of a row's split partials, in ascending split order with the
// log-sum-exp update: the arithmetic of decode attention without a window.
struct MergeParams {
  const float* ws_o;   // [rows][Hq][S][D]
  const float* ws_ml;  // [rows][Hq][S][2]
  const int32_t* kv_len;
  __nv_bfloat16* out;  // [rows][Hq][D]
  int Hq, S, max_len;
  Window win;
  int* status;
};

// The same fold by the threads of a cluster, whose block s holds partial s at the
// shared address `at`: o [rows][D], then (m, l) [rows]; pairs < G, at most eight
// partials, out [G][D].
template <int D, int THREADS>
__device__ __forceinline__ void fold_cluster(uint32_t at, int rows, int G, int rank, int blocks, int count,
                                             __nv_bfloat16* out) {
  for (int idx = rank * THREADS + static_cast<int>(threadIdx.x); idx < G * D; idx += blocks * THREADS) {
    const int pair = idx / D;
    float mv[8], lv[8], ov[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (s < count) {
        const uint32_t from = map_to_rank(at, s);
        mv[s] = ld_dsmem_f32(from + (rows * D + 2 * pair) * 4);
        lv[s] = ld_dsmem_f32(from + (rows * D + 2 * pair + 1) * 4);
        ov[s] = ld_dsmem_f32(from + idx * 4);
      }
    }
    float m_acc = -INFINITY, l_acc = 0.f, o_acc = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (s < count) {
        const float m_new = fmaxf(m_acc, mv[s]);
        const float fa = ex2_approx(__fsub_rn(m_acc, m_new)), fc = ex2_approx(__fsub_rn(mv[s], m_new));
        l_acc = __fadd_rn(__fmul_rn(l_acc, fa), __fmul_rn(lv[s], fc));
        o_acc = __fadd_rn(__fmul_rn(o_acc, fa), __fmul_rn(ov[s], fc));
        m_acc = m_new;
      }
    }
    out[idx] = __float2bfloat16_rn(count > 0 ? __fdiv_rn(o_acc, l_acc) : 0.f);
  }
}

// One block per (query head, row); thread d folds column d.  A row whose length
// is outside [0, max_len] gets zeros (the split kernel leaves it out).
template <int D>
__global__ void window_merge_kernel(const MergeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, row = blockIdx.y, d = threadIdx.x;
  int len = p.kv_len[row];
  if (len < 0 || len > p.max_len) {
    if (d == 0 && p.status) atomicExch(p.status, DEV_ATTN_BAD_LENGTH);
    len = 0;
  }
  const int64_t pair = static_cast<int64_t>(row) * p.Hq + h;
  __nv_bfloat16* dst = p.out + pair * D + d;
  if (len == 0) {
    *dst = __float2bfloat16_rn(0.f);
    return;
  }
  const int ns = visible_splits(p.win, window_lo(p.win, len), len).count;
  const float* o = p.ws_o + pair * p.S * D + d;
  const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + pair * p.S;
  float m_acc = -INFINITY, l_acc = 0.f, o_acc = 0.f;
  constexpr int CH = 16;  // partials loaded ahead of the (sequential) fold
  for (int s0 = 0; s0 < ns; s0 += CH) {
    float2 mlv[CH];
    float ov[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (s0 + i < ns) {
        mlv[i] = ml[s0 + i];
        ov[i] = o[static_cast<int64_t>(s0 + i) * D];
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (s0 + i < ns) {
        const float m_new = fmaxf(m_acc, mlv[i].x);
        const float fa = ex2_approx(__fsub_rn(m_acc, m_new));
        const float fc = ex2_approx(__fsub_rn(mlv[i].x, m_new));
        l_acc = __fadd_rn(__fmul_rn(l_acc, fa), __fmul_rn(mlv[i].y, fc));
        o_acc = __fadd_rn(__fmul_rn(o_acc, fa), __fmul_rn(ov[i], fc));
        m_acc = m_new;
      }
    }
  }
  *dst = __float2bfloat16_rn(__fdiv_rn(o_acc, l_acc));
}

// Of B rows; with a cache of no slots it is the whole call: zeros, and lengths that are
// not 0 reported.
template <int D>
inline kinv_status launch_window_merge(const MergeParams& p, int B, cudaStream_t stream) {
  return launch_kernel(window_merge_kernel<D>, dim3(p.Hq, B), dim3(D), 0, stream, 1, p);
}

}  // namespace kinv
