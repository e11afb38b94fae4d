// Log probabilities of given tokens, entropy and the likeliest alternatives of
// rows of logits (kinv_logprobs), one pass over the row.
//
// The row is cut into units of 1024 ids.  One warp takes a unit (32 ids a lane)
// and leaves, with m_u = max x and a = (x - m_u) log2 e,
//   S_u = sum 2^a,   T_u = sum 2^a a
// (a lane's ids in order on two chains, then a butterfly).  A row folds its
// units with M = max m_u and w_u = 2^((m_u - M) log2 e):  S = sum w_u S_u,
// T = sum w_u (T_u + S_u (m_u - M) log2 e), lane l of a warp the units l, l + 32,
// ... in order, then a butterfly; ln S, x - M - ln S and the entropy ln S -
// ln 2 T / S follow.  Which warp or block takes a unit changes nothing.  a is
// clamped at -200, so NaN (dropped by the maximum) and -infinity weigh 2^-200
// -> 0 and the product 2^a a stays finite.
//
// The k likeliest ids: every warp keeps its 32 best as 64-bit keys (the logit's
// ordered bits, then the complement of the id: larger is better and no two are
// equal), one per lane in descending order.  An id enters only if its logit
// reaches a floor that k ids are known to reach (from the block's first units,
// then from the best k of any of its warps) and its key beats the warp's k-th;
// entrants wait in shared memory and are merged 32 at a time by a bitonic
// network.  The lists of the warps and blocks of a row are merged the same way,
// and the result does not depend on the order, since the keys are distinct.
//
// What bounds it: issue slots and the exponentials (about 7 instructions and one
// ex2 per fp32 id, 6 per bf16 id).  4,096 bf16 rows of 151,936: 222 us, 5.6 TB/s
// (235 with every id widened and clamped on its own); units brought three ahead
// through shared memory instead of one ahead in registers were slower.
//
// A row is one block; a cluster of up to eight when there are few rows, or, where
// there are many short ones, a warp.  A cluster's blocks put their units' sums and
// their list into the first block's shared memory, so nothing goes through global
// memory.
#include <math.h>

#include "common.cuh"

namespace kinv {
namespace {

constexpr int DEV_LOGPROBS_BAD_ID = dev_code(9, KINV_ERR_INVALID_ARG);
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 1024;
constexpr int kPerLane = kUnit / 32;
constexpr int kMaxTop = 32;
constexpr int kPending = 64;
constexpr float kLog2e = 1.4426950408889634f;
// With the maximum of a unit of bf16 below this in magnitude, its ids may be raised to
// -2e30 in pairs: NaN and -infinity are finite then, and 2^a is 0 as with a = -200.
constexpr float kEasy = 1e30f;
constexpr float kLn2 = 0.6931471805599453f;

typedef unsigned long long u64;

struct LogprobParams {
  const void* x;
  int64_t ld;
  int rows, V, units;
  int parts, units_per_part;  // a row is `parts` blocks of `units_per_part` units
  const int32_t* ids;
  int n_ids;
  float* logprob;
  float* entropy;
  int top_k;
  int32_t* top_ids;
  float* top_logprobs;
  int* status;
};

__device__ __forceinline__ float no_nan(float x) { return x != x ? -INFINITY : x; }
// b - m of both halves, the bf16 operands as they are (mixed-precision fma).
__device__ __forceinline__ float2 less_m(__nv_bfloat162 b, float m) {
  float2 r;
  asm("{\n\t.reg .b16 a, b, one;\n\tmov.b32 {a, b}, %2;\n\tmov.b16 one, 0x3F80;\n\t"
      "fma.rn.f32.bf16 %0, a, one, %3;\n\tfma.rn.f32.bf16 %1, b, one, %3;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(*reinterpret_cast<const uint32_t*>(&b)), "f"(-m));
  return r;
}
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
      const bool keep_max = ((lane & j) == 0) == ((lane & k) == 0);
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

// A lane's 32 logits of a unit as raw 32-bit words, in 16-byte groups 32 lanes
// apart: element e (counted over the lane's words) is id (e / W) 32 W + lane W
// + e % W of the unit, W = 16 bytes of elements.  Ids past V read as -infinity.
template <typename T>
__device__ __forceinline__ int unit_id(int lane, int e) {
  constexpr int W = 16 / sizeof(T);
  return (e / W) * 32 * W + lane * W + e % W;
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_unit(const T* row, int first, int V, uint32_t (&x)[kPerLane * sizeof(T) / 4]) {
  const int lane = threadIdx.x & 31;
  constexpr int W = 16 / sizeof(T);
  if (VEC && first + kUnit <= V) {
#pragma unroll
    for (int i = 0; i < kPerLane / W; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + first + (i * 32 + lane) * W));
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else if (!VEC && sizeof(T) == 2 && first > 0 && first + kUnit + W <= V) {
    // a row off the 16-byte grid: the two chunks that hold a lane's ids, both within
    // the row, moved into place (512 rows of 50,001: 19.8 us, 25.5 id by id; 15.4 for
    // 50,000)
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + first);
    const uint32_t off = at & 15;  // the same for the warp
    const uint4* p = reinterpret_cast<const uint4*>(at - off);
#pragma unroll
    for (int i = 0; i < kPerLane / W; ++i) {
      const uint4 a = __ldg(p + i * 32 + lane), b = __ldg(p + i * 32 + lane + 1);
      uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 6; ++j) w[j] = off & 8 ? w[j + 2] : w[j];
#pragma unroll
      for (int j = 0; j < 5; ++j) w[j] = off & 4 ? w[j + 1] : w[j];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * i + j] = __funnelshift_r(w[j], w[j + 1], off & 2 ? 16 : 0);
    }
  } else {
#pragma unroll
    for (int w = 0; w < kPerLane * static_cast<int>(sizeof(T)) / 4; ++w) {
      if (sizeof(T) == 4) {
        const int id = first + unit_id<T>(lane, w);
        x[w] = id < V ? reinterpret_cast<const uint32_t*>(row)[id] : 0xFF800000u;
      } else {
        const int id = first + unit_id<T>(lane, 2 * w);
        const uint16_t* r16 = reinterpret_cast<const uint16_t*>(row);
        x[w] = (id < V ? r16[id] : 0xFF80u) | (id + 1 < V ? r16[id + 1] : 0xFF80u) << 16;
      }
    }
  }
}
// Elements 2i and 2i + 1 of a lane's words.
template <typename T, int N>
__device__ __forceinline__ float2 pair_of(const uint32_t (&x)[N], int i) {
  return sizeof(T) == 4 ? make_float2(__uint_as_float(x[2 * i % N]), __uint_as_float(x[(2 * i + 1) % N]))
                        : make_float2(bf16_lo(x[i % N]), bf16_hi(x[i % N]));
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

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// The lists of `n` warps of a row in shared memory, merged pairwise; the first of
// them returns the result.  Called by every thread of the block after the lists
// were written (no barrier yet); w: the warp's place among its row's.
__device__ __forceinline__ u64 merge_lists(u64 (*lists)[32], int n, int w) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  u64 v = lists[warp][lane];
#pragma unroll
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    if (half >= n) continue;
    __syncthreads();
    if (w < half) {
      v = merge_desc(lists[warp][lane], lists[warp + half][lane]);
      lists[warp][lane] = v;
    }
  }
  return v;
}

// WPR warps of a block (8 or 1), or a cluster of p.parts blocks, per row.
template <typename T, bool VEC, int WPR>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 4) logprobs_kernel(const LogprobParams p) {
  constexpr int N = kPerLane * sizeof(T) / 4;
  extern __shared__ float s_units[];  // per row of the block [units][3]: m, S, T (a cluster's: in its first block)
  __shared__ u64 pending[kWarps][kPending];
  __shared__ u64 lists[kWarps][32];
  __shared__ uint32_t s_first[kWarps];
  __shared__ uint32_t s_floor[kWarps];
  __shared__ float s_row[kWarps][2];
  if (threadIdx.x < kWarps) s_floor[threadIdx.x] = 0;
  if (p.parts > 1) cluster_arrive_relaxed();  // the first block runs: its shared memory may be written
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int wpr = WPR;
  const int w = warp & (wpr - 1), mine = warp - w;  // the row's first warp names it in the block
  const int part = blockIdx.x % p.parts;
  auto row_of = [&]() { return static_cast<int64_t>(blockIdx.x / p.parts) * (kWarps / wpr) + warp / wpr; };
  const bool live = row_of() < p.rows;
  const T* row = static_cast<const T*>(p.x) + (live ? row_of() : 0) * p.ld;
  const int u_end = live ? min(p.units, (part + 1) * p.units_per_part) : 0;
  const int top_k = p.top_k;
  u64 best = 0;  // lane i: the i-th best key (0: none)
  u64 bar = 0;   // the k-th best
  uint32_t floor_hi = 0;
  int waiting = 0;
  auto merge_waiting = [&](int n) {  // the last n entrants
    const u64 v = lane < n ? pending[warp][waiting - n + lane] : static_cast<u64>(0);
    __syncwarp();
    best = merge_desc(best, sort_desc(v));
    waiting -= n;
    bar = __shfl_sync(0xffffffffu, best, top_k - 1);
    if (lane == 0) atomicMax(&s_floor[mine], static_cast<uint32_t>(bar >> 32));
  };
  uint32_t x[N];
  int u = part * p.units_per_part + w;
  if (u < u_end) load_unit<T, VEC>(row, u * kUnit, p.V, x);
  const uint32_t unit_base = smem_addr(s_units) + warp / wpr * p.units * 12;
  if (p.parts > 1) cluster_wait();
  const uint32_t unit_dst = p.parts > 1 ? map_to_rank(unit_base, 0) : unit_base;
  bool first = true;
  // the block's warps take the same number of turns (a barrier in the first)
  for (; first || u < u_end; u += wpr) {
    uint32_t nx[N];
    const bool here = u < u_end;
    if (u + wpr < u_end) load_unit<T, VEC>(row, (u + wpr) * kUnit, p.V, nx);
    float lm = -INFINITY;
    if (here) {
      if (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; i += 2) lm = fmax3(lm, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
      } else {
        __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&x[0]);
#pragma unroll
        for (int i = 1; i < N; ++i) b = __hmax2(b, *reinterpret_cast<const __nv_bfloat162*>(&x[i]));
        lm = fmaxf(__low2float(b), __high2float(b));
      }
      lm = no_nan(lm);
    }
    if (first && top_k > 0) {
      // with n of the row's warps holding a unit and q = ceil(k / n): each warp's
      // q-th largest lane maximum; the ceil(k / q)-th largest of those is reached
      // by at least k ids
      const int n = max(1, min(wpr, u_end - part * p.units_per_part));
      const int q = (top_k + n - 1) / n, need = (top_k + q - 1) / q;
      const uint32_t kth = __shfl_sync(0xffffffffu, sort_desc(here ? ordered(lm) : 0u), q - 1);
      if (lane == 0) s_first[warp] = kth;
      __syncthreads();
      const int me = lane & (wpr - 1);
      const uint32_t v = s_first[mine + me];
      int rank = 0;
#pragma unroll
      for (int o = 0; o < wpr; ++o) {
        const uint32_t other = s_first[mine + o];
        rank += other > v || (other == v && o < me);
      }
      floor_hi = __shfl_sync(0xffffffffu, v, __ffs(__ballot_sync(0xffffffffu, rank == need - 1)) - 1);
    }
    first = false;
    if (!here) break;
    const float m = warp_max(lm);
    float s = 0.f, t = 0.f;
    if (m == INFINITY) {  // the ids at +infinity share the row
#pragma unroll
      for (int i = 0; i < kPerLane / 2; ++i) {
        const float2 v = pair_of<T>(x, i);
        s += (v.x == INFINITY ? 1.f : 0.f) + (v.y == INFINITY ? 1.f : 0.f);
      }
    } else if (sizeof(T) == 2 && fabsf(m) < kEasy) {
      // the same values: what is raised here weighs 0 either way
      const float2 c2 = make_float2(kLog2e, kLog2e);
      const __nv_bfloat162 low = __float2bfloat162_rn(-2.f * kEasy);
      float2 s2 = make_float2(0.f, 0.f), t2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kPerLane / 2; ++i) {
        const __nv_bfloat162 b = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x[i % N]), low);
        const float2 a = __fmul2_rn(less_m(b, m), c2);
        const float2 w = make_float2(ex2_approx(a.x), ex2_approx(a.y));
        s2 = __fadd2_rn(s2, w);
        t2 = __ffma2_rn(w, a, t2);
      }
      s = __fadd_rn(s2.x, s2.y);
      t = __fadd_rn(t2.x, t2.y);
    } else if (m > -INFINITY) {
      const float2 neg_m = make_float2(-m, -m), c2 = make_float2(kLog2e, kLog2e);
      float2 s2 = make_float2(0.f, 0.f), t2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kPerLane / 2; ++i) {
        float2 a = __fmul2_rn(__fadd2_rn(pair_of<T>(x, i), neg_m), c2);
        a = make_float2(fmaxf(a.x, -200.f), fmaxf(a.y, -200.f));
        const float2 w = make_float2(ex2_approx(a.x), ex2_approx(a.y));
        s2 = __fadd2_rn(s2, w);
        t2 = __ffma2_rn(w, a, t2);
      }
      s = __fadd_rn(s2.x, s2.y);
      t = __fadd_rn(t2.x, t2.y);
    }
    s = warp_sum(s);
    t = warp_sum(t);
    if (lane < 3) st_cluster_f32(unit_dst + (3 * u + lane) * 4, lane == 0 ? m : lane == 1 ? s : t);
    if (top_k > 0) {
      floor_hi = max(floor_hi, *static_cast<volatile uint32_t*>(&s_floor[mine]));
      if (__any_sync(0xffffffffu, ordered(lm) >= floor_hi)) {
        // which of the lane's ids reach the floor; then one id a lane at a time
        const float floor = floor_hi ? unordered(floor_hi) : -INFINITY;
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < kPerLane / 2; ++i) {
          const float2 v = pair_of<T>(x, i);
          mask |= (v.x < floor ? 0u : 1u << (2 * i)) | (v.y < floor ? 0u : 2u << (2 * i));
        }
        while (__any_sync(0xffffffffu, mask != 0)) {
          u64 key = 0;
          if (mask) {
            const int id = u * kUnit + unit_id<T>(lane, __ffs(mask) - 1);
            mask &= mask - 1;
            if (id < p.V) key = top_key(static_cast<float>(row[id]), id);
          }
          const bool in = key > bar;
          const unsigned who = __ballot_sync(0xffffffffu, in);
          if (in) pending[warp][waiting + __popc(who & ((1u << lane) - 1))] = key;
          waiting += __popc(who);
          __syncwarp();
          if (waiting >= 32) merge_waiting(32);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = nx[i];
  }
  // the row's list and sums to the first block
  if (top_k > 0) {
    if (waiting) merge_waiting(waiting);
    lists[warp][lane] = best;
    best = merge_lists(lists, wpr, w);
  }
  if (p.parts > 1) {
    if (top_k > 0) {
      // the other blocks' lists go where the first block's `pending` was (its
      // own warps are past it: the merge's barriers above, then the cluster's)
      if (warp == 0) lists[0][lane] = best;
      cluster_sync();
      if (part != 0) {
        if (warp == 0) st_cluster_u64(map_to_rank(smem_addr(&pending[0][0]), 0) + (part * 32 + lane) * 8, best);
      }
    }
    cluster_sync();
    if (part != 0) return;
    if (top_k > 0) {
      u64(*got)[32] = reinterpret_cast<u64(*)[32]>(&pending[0][0]);
      const u64 v = warp == 0 ? lists[0][lane] : warp < p.parts ? got[warp][lane] : static_cast<u64>(0);
      __syncthreads();
      lists[warp][lane] = v;
      best = merge_lists(lists, kWarps, warp);
    }
  }
  __syncthreads();
  const int64_t r = row_of();
  const float* s_unit = s_units + warp / wpr * p.units * 3;
  // the fold of the units, by the row's last warp
  if (w == wpr - 1 && live) {
    float M = -INFINITY;
    for (int i = lane; i < p.units; i += 32) M = fmaxf(M, s_unit[3 * i]);
    M = warp_max(M);
    float S = 0.f, Tt = 0.f;
    for (int i = lane; i < p.units; i += 32) {
      const float m = s_unit[3 * i], s = s_unit[3 * i + 1], t = s_unit[3 * i + 2];
      const float d = m == M ? 0.f : __fmul_rn(__fsub_rn(m, M), kLog2e);
      const float w = ex2_approx(d);
      if (w > 0.f) {
        S = __fadd_rn(S, __fmul_rn(w, s));
        Tt = __fadd_rn(Tt, __fmul_rn(w, __fmaf_rn(s, d, t)));
      }
    }
    S = warp_sum(S);
    Tt = warp_sum(Tt);
    if (lane == 0) {
      const float ln_s = logf(S);
      s_row[mine][0] = M;
      s_row[mine][1] = ln_s;
      if (p.entropy) p.entropy[r] = M == -INFINITY ? 0.f : __fsub_rn(ln_s, __fmul_rn(kLn2, __fdiv_rn(Tt, S)));
    }
  }
  __syncthreads();
  if (!live) return;
  const float M = s_row[mine][0], ln_s = s_row[mine][1];
  auto logprob = [&](float v) {
    v = no_nan(v);
    if (M == -INFINITY) return -INFINITY;
    const float d = v == M ? 0.f : __fsub_rn(v, M);  // +infinity against +infinity: the shared maximum
    return __fsub_rn(d, ln_s);
  };
  if (w == 0 && lane < top_k) {
    p.top_ids[r * top_k + lane] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
    p.top_logprobs[r * top_k + lane] = logprob(unordered(static_cast<uint32_t>(best >> 32)));
  }
  for (int j = w * 32 + lane; j < p.n_ids; j += wpr * 32) {
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
}

// Blocks per row: one for every SM, while each keeps a unit per warp (256 fp32
// rows with 20 alternatives: 37 us as 256 blocks, 46 as 512, 54 as 1,024; one row:
// 22 us as one block, 9 as eight).
int part_count(int rows, int units) {
  int parts = 1;
  while (parts < 8 && static_cast<int64_t>(rows) * parts < sm_count() && units > parts * kWarps) parts *= 2;
  return parts;
}

template <typename T, int WPR>
kinv_status launch(const LogprobParams& p, bool vec, cudaStream_t stream) {
  constexpr int ROWS = kWarps / WPR;  // of a block
  const size_t smem = static_cast<size_t>(p.units) * 12 * ROWS;
  auto* kernel = vec ? logprobs_kernel<T, true, WPR> : logprobs_kernel<T, false, WPR>;
  const kinv_status attr = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
  if (attr != KINV_OK) return attr;
  const int64_t blocks = (static_cast<int64_t>(p.rows) + ROWS - 1) / ROWS * p.parts;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), smem, stream, p.parts, p);
}

// A warp per row where a block's eight would not have a unit each and the rows
// alone fill the SMs with sixteen warps (4,096 rows of 5,000 fp32 with 20
// alternatives: 34 us, 76 with eight warps a row; 8,192 rows of 500: 25 and 135).
template <typename T>
kinv_status launch(const LogprobParams& p, bool vec, cudaStream_t stream) {
  return p.units <= kWarps && p.rows >= sm_count() * 16 ? launch<T, 1>(p, vec, stream) : launch<T, kWarps>(p, vec, stream);
}

}  // namespace
}  // namespace kinv

using namespace kinv;

extern "C" kinv_status kinv_logprobs(const void* logits, kinv_dtype dtype, int64_t ld, int rows, int V,
                                     const int32_t* ids, int n_ids, float* logprob, float* entropy, int top_k,
                                     int32_t* top_ids, float* top_logprobs, kinv_stream stream) {
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
  p.rows = rows;
  p.V = V;
  p.units = (V + kUnit - 1) / kUnit;
  p.parts = part_count(rows, p.units);
  p.units_per_part = (p.units + p.parts - 1) / p.parts;
  p.ids = ids;
  p.n_ids = n_ids;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_k = top_k;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  p.status = device_status_word();
  const bool vec = aligned16(logits) && static_cast<size_t>(ld) * elem % 16 == 0;
  return dtype == KINV_F32 ? launch<float>(p, vec, stream) : launch<__nv_bfloat16>(p, vec, stream);
}
