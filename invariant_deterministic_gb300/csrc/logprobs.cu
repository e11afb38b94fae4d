// Log probabilities of given tokens, entropy and the likeliest alternatives of
// rows of logits (kinv_logprobs), one pass over the row.
//
// The row is cut into units of 512 ids.  One warp takes a unit (16 ids a lane)
// and leaves, with m_u = max x and a = (x - m_u) log2 e,
//   S_u = sum 2^a,   T_u = sum 2^a a
// a lane's ids in order, then a butterfly.  A row folds its units with M =
// max m_u and w_u = 2^((m_u - M) log2 e):  S = sum w_u S_u,  T = sum w_u (T_u +
// S_u (m_u - M) log2 e), lane l of a warp the units l, l + 32, ... in order,
// then a butterfly; ln S, x - M - ln S and the entropy ln S - ln 2 T / S follow.
// Which warp or block takes a unit changes nothing.  a is clamped at -200, so
// NaN (dropped by the maximum) and -infinity weigh 2^-200 -> 0 and the product
// 2^a a stays finite.
//
// The k likeliest ids: every warp keeps its 32 best as 64-bit keys (the logit's
// ordered bits, then the complement of the id: larger is better and no two are
// equal), one per lane in descending order.  An id enters only if its key beats
// the k-th; entrants wait in shared memory and are merged 32 at a time by a
// bitonic network.  The lists of the warps and blocks of a row are merged the
// same way, and the result does not depend on the order, since the keys are
// distinct.
#include <math.h>

#include "common.cuh"

namespace kinv {
namespace {

constexpr int DEV_LOGPROBS_BAD_ID = dev_code(9, KINV_ERR_INVALID_ARG);
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 512;
constexpr int kMaxTop = 32;
constexpr int kPending = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef unsigned long long u64;

struct LogprobParams {
  const void* x;
  int64_t ld;
  int V, units, parts, units_per_part;  // a row is `parts` blocks of `units_per_part` units
  const int32_t* ids;
  int n_ids;
  float* logprob;
  float* entropy;
  int top_k;
  int32_t* top_ids;
  float* top_logprobs;
  float* ws_unit;  // [rows][units][3]: m, S, T
  u64* ws_top;     // [rows][parts][32]
  int* status;
};

__device__ __forceinline__ float no_nan(float x) { return x != x ? -INFINITY : x; }
// Unsigned integers in the order of the floats (-0 as +0, NaN as -infinity).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(no_nan(x), 0.f));
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ u64 top_key(float x, int id) {
  return static_cast<u64>(ordered(x)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

// The 32 lanes' values in descending order, lane 0 the largest.
template <typename T>
__device__ __forceinline__ T sort_desc(T v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const T o = __shfl_xor_sync(0xffffffffu, v, j);
      const bool keep_max = ((lane & j) == 0) == ((lane & k) == 0 || k == 32);
      v = keep_max ? (v > o ? v : o) : (v < o ? v : o);
    }
  }
  return v;
}
// The 32 largest of two descending lists, descending.
__device__ __forceinline__ u64 merge_desc(u64 a, u64 b) {
  const int lane = threadIdx.x & 31;
  const u64 r = __shfl_sync(0xffffffffu, b, 31 - lane);
  u64 v = a > r ? a : r;  // bitonic
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const u64 o = __shfl_xor_sync(0xffffffffu, v, j);
    v = (lane & j) == 0 ? (v > o ? v : o) : (v < o ? v : o);
  }
  return v;
}

// A lane's 16 logits of a unit.  fp32: x[4 i + j] is id 128 i + 4 lane + j;
// bf16: x[8 i + j] is id 256 i + 8 lane + j.  Ids past V read as -infinity.
template <typename T>
__device__ __forceinline__ int unit_id(int lane, int e) {
  constexpr int W = 16 / sizeof(T);
  return (e / W) * 32 * W + lane * W + e % W;
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_unit(const T* row, int first, int V, float (&x)[16]) {
  const int lane = threadIdx.x & 31;
  constexpr int W = 16 / sizeof(T);
  if (VEC && first + kUnit <= V) {
#pragma unroll
    for (int i = 0; i < 16 / W; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + first + (i * 32 + lane) * W);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4) {
          x[4 * i + j] = __uint_as_float(w[j]);
        } else {
          x[(8 * i + 2 * j) & 15] = bf16_lo(w[j]);
          x[(8 * i + 2 * j + 1) & 15] = bf16_hi(w[j]);
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int id = first + unit_id<T>(lane, e);
      x[e] = id < V ? static_cast<float>(row[id]) : -INFINITY;
    }
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Results of a row from its units' sums and its 32 best keys (lane i the
// i-th); one warp.
template <typename T>
__device__ void finish_row(const LogprobParams& p, int64_t r, const float* unit, u64 best) {
  const int lane = threadIdx.x & 31;
  float M = -INFINITY;
  for (int u = lane; u < p.units; u += 32) M = fmaxf(M, unit[3 * u]);
  M = warp_max(M);
  float S = 0.f, Tt = 0.f;
  for (int u = lane; u < p.units; u += 32) {
    const float m = unit[3 * u], s = unit[3 * u + 1], t = unit[3 * u + 2];
    const float d = m == M ? 0.f : __fmul_rn(__fsub_rn(m, M), kLog2e);
    const float w = ex2_approx(d);
    if (w > 0.f) {
      S = __fadd_rn(S, __fmul_rn(w, s));
      Tt = __fadd_rn(Tt, __fmul_rn(w, __fmaf_rn(s, d, t)));
    }
  }
  S = warp_sum(S);
  Tt = warp_sum(Tt);
  const float ln_s = logf(S);
  auto logprob = [&](float x) {
    x = no_nan(x);
    if (M == -INFINITY) return -INFINITY;
    const float d = x == M ? 0.f : __fsub_rn(x, M);  // +infinity against +infinity: the shared maximum
    return __fsub_rn(d, ln_s);
  };
  const T* row = static_cast<const T*>(p.x) + r * p.ld;
  if (lane == 0 && p.entropy)
    p.entropy[r] = M == -INFINITY ? 0.f : __fsub_rn(ln_s, __fmul_rn(kLn2, __fdiv_rn(Tt, S)));
  for (int j = lane; j < p.n_ids; j += 32) {
    const int id = p.ids[r * p.n_ids + j];
    float v = 0.f;
    if (id >= p.V) {
      v = __int_as_float(0x7fffffff);
      if (p.status) atomicExch(p.status, DEV_LOGPROBS_BAD_ID);
    } else if (id >= 0) {
      v = logprob(static_cast<float>(row[id]));
    }
    p.logprob[r * p.n_ids + j] = v;
  }
  if (lane < p.top_k) {
    p.top_ids[r * p.top_k + lane] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
    p.top_logprobs[r * p.top_k + lane] = logprob(unordered(static_cast<uint32_t>(best >> 32)));
  }
}

// The block's lists in shared memory, one per warp, into one (warp 0).
__device__ __forceinline__ u64 merge_block(u64 (*lists)[32], u64 mine) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  lists[warp][lane] = mine;
  __syncthreads();
  if (warp == 0) {
#pragma unroll 1
    for (int w = 1; w < kWarps; ++w) mine = merge_desc(mine, lists[w][lane]);
  }
  return mine;
}

// A block per (part of a row, row).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobParams p) {
  extern __shared__ float s_unit[];  // [units][3] when the row is one part
  __shared__ u64 pending[kWarps][kPending];
  __shared__ u64 lists[kWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t r = blockIdx.x / p.parts;
  const int part = blockIdx.x % p.parts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(p.x) + r * p.ld;
  float* unit = p.parts == 1 ? s_unit : p.ws_unit + r * p.units * 3;
  const int u_end = min(p.units, (part + 1) * p.units_per_part);
  u64 best = 0;   // lane i: the i-th best key (0: none)
  u64 bar = 0;    // the k-th best
  uint32_t bar_hi = 0;
  int waiting = 0;
  bool first = true;
  for (int u = part * p.units_per_part + warp; u < u_end; u += kWarps) {
    float x[16];
    load_unit<T, VEC>(row, u * kUnit, p.V, x);
    float lm = x[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) lm = fmaxf(lm, x[e]);
    lm = no_nan(lm);
    const float m = warp_max(lm);
    float s = 0.f, t = 0.f;
    if (m == INFINITY) {  // the ids at +infinity share the row
#pragma unroll
      for (int e = 0; e < 16; ++e) s += x[e] == INFINITY ? 1.f : 0.f;
    } else if (m > -INFINITY) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float a = fmaxf(__fmul_rn(__fsub_rn(x[e], m), kLog2e), -200.f);
        const float w = ex2_approx(a);
        s = __fadd_rn(s, w);
        t = __fmaf_rn(w, a, t);
      }
    }
    s = warp_sum(s);
    t = warp_sum(t);
    if (lane == 0) {
      unit[3 * u] = m;
      unit[3 * u + 1] = s;
      unit[3 * u + 2] = t;
    }
    if (p.top_k > 0) {
      uint32_t floor_hi = bar_hi;
      if (first) {
        // k lanes hold an id at or above the k-th of the lanes' maxima
        floor_hi = __shfl_sync(0xffffffffu, sort_desc(ordered(lm)), p.top_k - 1);
      }
      if (__any_sync(0xffffffffu, ordered(lm) >= floor_hi)) {
#pragma unroll 1
        for (int e0 = 0; e0 < 16; e0 += 4) {
#pragma unroll
          for (int e1 = 0; e1 < 4; ++e1) {
            float xe = x[e1];
#pragma unroll
            for (int q = 1; q < 4; ++q) xe = e0 == 4 * q ? x[4 * q + e1] : xe;
            const int id = u * kUnit + unit_id<T>(lane, e0 + e1);
            const u64 key = id < p.V ? top_key(xe, id) : 0;
            const bool in = key > bar && static_cast<uint32_t>(key >> 32) >= floor_hi;
            const unsigned who = __ballot_sync(0xffffffffu, in);
            if (who) {
              if (in) pending[warp][waiting + __popc(who & ((1u << lane) - 1))] = key;
              waiting += __popc(who);
              __syncwarp();
              if (waiting >= 32) {
                best = merge_desc(best, sort_desc(pending[warp][waiting - 32 + lane]));
                waiting -= 32;
                bar = __shfl_sync(0xffffffffu, best, p.top_k - 1);
                __syncwarp();
              }
            }
          }
        }
        if (first && waiting) {
          const u64 v = lane < waiting ? pending[warp][lane] : 0;
          best = merge_desc(best, sort_desc(v));
          bar = __shfl_sync(0xffffffffu, best, p.top_k - 1);
          waiting = 0;
          __syncwarp();
        }
        bar_hi = static_cast<uint32_t>(bar >> 32);
      }
      first = false;
    }
  }
  if (p.top_k > 0) {
    if (waiting) best = merge_desc(best, sort_desc(lane < waiting ? pending[warp][lane] : static_cast<u64>(0)));
    best = merge_block(lists, best);
  } else {
    __syncthreads();
  }
  if (warp != 0) return;
  if (p.parts == 1)
    finish_row<T>(p, r, s_unit, best);
  else if (p.top_k > 0)
    p.ws_top[(r * p.parts + part) * 32 + lane] = best;
}

// Rows of several parts: a block per row.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_finish_kernel(const LogprobParams p) {
  __shared__ u64 lists[kWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t r = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  u64 best = 0;
  if (p.top_k > 0) {
    for (int part = warp; part < p.parts; part += kWarps)
      best = merge_desc(best, p.ws_top[(r * p.parts + part) * 32 + lane]);
    best = merge_block(lists, best);
  }
  if (warp == 0) finish_row<T>(p, r, p.ws_unit + r * p.units * 3, best);
}

int part_count(int rows, int units) {
  const int most = (units + kWarps - 1) / kWarps;
  const int want = (152 * 4 + rows - 1) / rows;
  return want < most ? want : most;
}

size_t unit_bytes(int rows, int units) { return (static_cast<size_t>(rows) * units * 12 + 255) / 256 * 256; }

template <typename T>
kinv_status launch(const LogprobParams& p, int rows, bool vec, cudaStream_t stream) {
  const size_t smem = p.parts == 1 ? static_cast<size_t>(p.units) * 12 : 0;
  auto* kernel = vec ? logprobs_kernel<T, true> : logprobs_kernel<T, false>;
  const kinv_status attr = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
  if (attr != KINV_OK) return attr;
  const kinv_status st = launch_kernel(kernel, dim3(static_cast<unsigned>(rows) * p.parts), dim3(kThreads), smem, stream, 1, p);
  if (st != KINV_OK || p.parts == 1) return st;
  return launch_kernel(logprobs_finish_kernel<T>, dim3(rows), dim3(kThreads), 0, stream, 1, p);
}

}  // namespace
}  // namespace kinv

using namespace kinv;

extern "C" size_t kinv_logprobs_workspace(int rows, int V) {
  if (rows <= 0 || V <= 0) return 0;
  const int units = (V + kUnit - 1) / kUnit;
  const int parts = part_count(rows, units);
  return parts == 1 ? 0 : unit_bytes(rows, units) + static_cast<size_t>(rows) * parts * 32 * 8;
}

extern "C" kinv_status kinv_logprobs(const void* logits, kinv_dtype dtype, int64_t ld, int rows, int V,
                                     const int32_t* ids, int n_ids, float* logprob, float* entropy, int top_k,
                                     int32_t* top_ids, float* top_logprobs, void* workspace,
                                     size_t workspace_bytes, kinv_stream stream) {
  if (rows < 0 || V <= 0 || n_ids < 0 || top_k < 0 || ld < V || top_k > V) return KINV_ERR_INVALID_ARG;
  if (dtype != KINV_F32 && dtype != KINV_BF16) return KINV_ERR_INVALID_ARG;
  if (V > 1048576 || top_k > kMaxTop) return KINV_ERR_UNSUPPORTED;
  if (rows == 0) return KINV_OK;
  if (!logits || (n_ids > 0 && (!ids || !logprob)) || (top_k > 0 && (!top_ids || !top_logprobs)))
    return KINV_ERR_INVALID_ARG;
  const size_t elem = dtype == KINV_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % elem) return KINV_ERR_ALIGNMENT;
  LogprobParams p{};
  p.x = logits;
  p.ld = ld;
  p.V = V;
  p.units = (V + kUnit - 1) / kUnit;
  p.parts = part_count(rows, p.units);
  p.units_per_part = (p.units + p.parts - 1) / p.parts;
  if (static_cast<int64_t>(rows) * p.parts > 0x7fffffff) return KINV_ERR_UNSUPPORTED;
  const size_t need = kinv_logprobs_workspace(rows, V);
  if (need > 0) {
    if (!workspace) return KINV_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return KINV_ERR_ALIGNMENT;
    if (workspace_bytes < need) return KINV_ERR_WORKSPACE;
    p.ws_unit = static_cast<float*>(workspace);
    p.ws_top = reinterpret_cast<u64*>(static_cast<char*>(workspace) + unit_bytes(rows, p.units));
  }
  p.ids = ids;
  p.n_ids = n_ids;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_k = top_k;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  p.status = device_status_word();
  const bool vec = aligned16(logits) && static_cast<size_t>(ld) * elem % 16 == 0;
  return dtype == KINV_F32 ? launch<float>(p, rows, vec, stream) : launch<__nv_bfloat16>(p, rows, vec, stream);
}
