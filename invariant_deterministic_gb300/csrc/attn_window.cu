// Prefill attention with a sliding window and sinks (window 0: every key), on the
// tcgen05 tensor cores.
//
// Per (row, head) pair the arithmetic is kinv_attn_decode's (see attention.cu):
// 256-key splits at absolute offsets, R = Q . K^T in 16-deep steps, base-2 softmax
// weights carried as bf16 hi and lo, one fp32 chain of sixteen 16-key steps, the
// splits folded left to right with every product and sum rounded on its own.  So
// a row has the bits of the decode step at its position.
//
// Work: tiles of 128 pairs of one sequence and kv head (128 / G rows), each with
// the list of splits that hold a key one of its rows sees.  A block stays on its
// SM and walks its tiles, longest first, and their splits as one sequence of
// steps, so that a tile's first copies and products run beside the last softmax of
// the tile before (a block per tile left about 5 of 31 us between tiles of six
// splits).
//
// Few tiles over many splits (a short chunk behind a long context) would leave most
// SMs without work, and a row's fold is one chain.  There (PARTS) the steps of all tiles
// are dealt to the blocks in equal runs, counted on the device; a step leaves its
// partial in the workspace, columns by pairs so that a warp's stores are whole lines,
// and prefill_fold_kernel folds the partials in the same order: the same bits.
//
// Roles (608 threads).  Warps 0-15: four threads per pair (TMEM lane = pair),
// quarter w / 4 taking the 32-key groups w / 4 and w / 4 + 4 of each split and D / 4
// columns of the fold; they exchange raw maxima and 32-key sums through shared
// memory.  Warp 16 issues the MMAs and owns tensor memory; warp 17 issues the copies
// of Q and K, warp 18 those of V, and zeroes V rows that no row of the tile sees (a
// weight of 0 times a NaN would not be 0).
//
// Tensor memory: three buffers of 128 columns for the halves of R, used in turn,
// and O.  A thread writes its groups' P over their R as packed bf16 pairs (sixteen
// keys at column c: hi at c, lo 8 columns further), read by the PV MMAs as their A
// operand.
// MMAs run in issue order: R(s + 1, half 0), PV(s, half 0), R(s + 1, half 1) over
// the buffer that these products read, PV(s, half 1).  So the next step's scores are
// there when its softmax begins, with half of this step's products beside it.  With
// R in two halves and O in two buffers instead, R waited for all of P . V: 7,500
// cycles a step.  The softmax threads fold step s - 1 between the two halves of
// their weights, when its products are done.
#include <math.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_mma.cuh"
#include "attn_tc.cuh"
#include "common.cuh"
#include "window.cuh"

namespace kinv {
namespace {

constexpr int kSplit = kSplitKeys;
constexpr int kPairs = 128;
constexpr int kSoftmax = 512;
constexpr int kThreads = kSoftmax + 96;
constexpr int kBars = 19;

struct Args {
  const int32_t* q_start;
  const int32_t* q_len;
  const int32_t* q_offset;
  __nv_bfloat16* out;
  int B, Hq, Hkv, G, RT;  // RT rows per tile (128 / G)
  int tiles_per_seq;
  int max_len, max_q_len, total_rows;
  float c2;               // fp32(scale * log2 e) > 0
  int* status;
  Window win;
  float* parts;           // PARTS: [step][D / 4][128 pairs][4] ...
  float2* parts_ml;       // ... and (m, l), [step][128 pairs]
};

// At most this many tiles (a quarter of the SMs) are spread over the GPU, from this many
// splits on.  32/8 heads of 128, whole tiles against spread: 16 rows behind 300 keys
// (two splits) 16.6 and 16.5 us, behind 600 20.6 and 16.5, 8,000 108 and 27, 32,000 392
// and 66; 128 rows (32 tiles) 20.6 and 19.5 behind 600, 109 and 53 behind 8,000; 256 rows
// (64 tiles) 112 and 110 there, with 134 MB of partials.
constexpr int kFewTiles = 38, kFewSplits = 3;

// One step of a block: a split of a tile.
struct Step {
  int b, g, row0, nrows, len0;  // rows of q / out; row r sees keys below len0 + r
  int lo, it, ns;               // the first row's first window key; step it of ns of the tile
  bool fresh;                   // the block's first step of the tile
  SplitList list;
  __device__ int k0() const { return list.split(it) * kSplit; }
  __device__ int len_last() const { return len0 + nrows - 1; }
};

// Tile `at` in the order of the walk (whose tiles get shorter), or false: a tile behind
// its sequence's rows, or a sequence whose device-side numbers break the stated bounds.
__device__ __forceinline__ bool tile_at(const Args& a, int at, Step& s) {
  const int per = a.Hkv * a.B, rank = at / per, rest = at - rank * per;
  const int tile = a.tiles_per_seq - 1 - rank;
  s.g = rest % a.Hkv;
  s.b = rest / a.Hkv;
  const int n = a.q_len[s.b], st0 = a.q_start[s.b], off = a.q_offset[s.b];
  if (!(n >= 0 && n <= a.max_q_len && st0 >= 0 && st0 <= a.max_len - n && off >= 0 && off <= a.total_rows - n)) {
    if (threadIdx.x == 0 && tile == 0 && a.status) atomicExch(a.status, DEV_ATTN_BAD_LENGTH);
    return false;
  }
  const int first = tile * a.RT;
  if (first >= n) return false;
  s.nrows = min(a.RT, n - first);
  s.row0 = off + first;
  s.len0 = st0 + first + 1;
  s.lo = window_lo(a.win, s.len0);
  s.list = visible_splits(a.win, s.lo, s.len_last());
  s.ns = s.list.count;
  return true;
}

__device__ __forceinline__ int lane_tile_splits(const Args& a, int at, int tiles) {
  Step s;
  return at < tiles && tile_at(a, at, s) ? s.ns : 0;
}

// The block's steps in order.  Round r of the blocks over the tiles runs forwards
// for even r, backwards for odd r: the tiles get shorter, and who had the longest
// of one round gets the shortest of the next.  PARTS: steps begin .. end - 1 of all
// tiles' steps one behind the other.
template <bool PARTS>
struct Walk {
  const Args& a;
  int round;           // PARTS: the tile
  int at_step, left;   // PARTS: the step among all tiles' steps; how many follow it
  Step s;
  __device__ explicit Walk(const Args& args) : a(args), round(0), at_step(0), left(0) {
    s.it = s.ns = 0;
    if (PARTS) {
      const int lane = threadIdx.x & 31, tiles = a.tiles_per_seq * a.Hkv * a.B;
      const int n0 = lane_tile_splits(a, lane, tiles), n1 = lane_tile_splits(a, lane + 32, tiles);
      int i0 = n0, i1 = n1;  // inclusive sums
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u0 = __shfl_up_sync(0xffffffffu, i0, o), u1 = __shfl_up_sync(0xffffffffu, i1, o);
        if (lane >= o) {
          i0 += u0;
          i1 += u1;
        }
      }
      i1 += __shfl_sync(0xffffffffu, i0, 31);
      const int64_t all = __shfl_sync(0xffffffffu, i1, 31);
      const int begin = static_cast<int>(all * blockIdx.x / gridDim.x);
      left = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x) - begin;
      // the tile that holds step `begin`: the first whose inclusive sum is above it
      const int tile = __popc(__ballot_sync(0xffffffffu, i0 <= begin)) + __popc(__ballot_sync(0xffffffffu, i1 <= begin));
      const int excl0 = __shfl_sync(0xffffffffu, i0 - n0, tile & 31), excl1 = __shfl_sync(0xffffffffu, i1 - n1, tile & 31);
      at_step = begin - 1;
      round = tile;
      if (left > 0) {
        tile_at(a, tile, s);
        s.it = begin - (tile < 32 ? excl0 : excl1) - 1;
        s.fresh = false;
        first = true;
      }
    }
  }
  bool first = false;  // PARTS: no step yet
  __device__ bool next() {
    if (PARTS) {
      if (left <= 0) return false;
      --left;
      ++at_step;
      s.fresh = first;
      first = false;
      if (++s.it < s.ns) return true;
      // a tile follows, for steps are left; without one (lengths written over while the
      // call runs) the walk ends
      const int tiles = a.tiles_per_seq * a.Hkv * a.B;
      do {
        if (++round >= tiles) {
          left = 0;
          return false;
        }
      } while (!tile_at(a, round, s));
      s.it = 0;
      s.fresh = true;
      return true;
    }
    s.fresh = false;
    if (++s.it < s.ns) return true;
    const int grid = gridDim.x, total = a.tiles_per_seq * a.Hkv * a.B;
    for (;; ++round) {
      if (static_cast<int64_t>(round) * grid >= total) return false;
      const int at = round * grid + (round & 1 ? grid - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
      if (at >= total || !tile_at(a, at, s)) continue;
      s.it = 0;
      s.fresh = true;
      ++round;
      return true;
    }
  }
};

template <int D, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prefill_window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                               const __grid_constant__ CUtensorMap tmV, const Args a) {
  constexpr int DS = D / 64;                   // 64-wide slices of the head dimension
  constexpr int Q_SLICE = kPairs * 128;        // [128 pairs][64]
  constexpr int Q_BYTES = DS * Q_SLICE;
  constexpr int KV_SLICE = kPairs * 128;       // [128 keys][64]: half a split
  constexpr int KV_BYTES = DS * KV_SLICE;
  constexpr int DQ = D / 4;                    // output columns per thread
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* q_s = base;
  unsigned char* k_s = q_s + Q_BYTES;          // three halves, used in turn
  unsigned char* v_s = k_s + 3 * KV_BYTES;     // both halves of a split
  float* x_max = reinterpret_cast<float*>(v_s + 2 * KV_BYTES);  // [2][4][128] raw maxima, by the step's parity
  float* x_w = x_max + 2 * 4 * kPairs;                           // [2][8][128] sums of 32 weights
  uint64_t* bars = reinterpret_cast<uint64_t*>(x_w + 2 * 8 * kPairs);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_addr(bars + i); };
  const uint32_t q_full = bar(0), s_full = bar(1), o_full = bar(2), o_free = bar(3), done_bar = bar(4);
  auto k_full = [&](int i) { return bar(5 + i % 3); };    // half i = 2 step + h
  auto k_empty = [&](int i) { return bar(8 + i % 3); };
  auto v_full = [&](int h) { return bar(11 + h); };
  auto v_ready = [&](int h) { return bar(13 + h); };
  auto v_empty = [&](int h) { return bar(15 + h); };
  auto p_full = [&](int h) { return bar(17 + h); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = threadIdx.x;
  if (t == 0) {
    for (int i = 0; i < kBars; ++i) {
      // o_free and p_full: all softmax threads; the rest one arrival (a thread or a commit)
      mbar_init(bar(i), i == 3 || i >= 17 ? kSoftmax : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 16) tmem_alloc(smem_addr(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // after the TMEM allocation (see the GEMM kernels)
  pdl_wait();
  int* status = a.status;
  Walk<PARTS> walk(a);

  if (warp == 17) {
    // ---- Q and K, as early as their place is free: K half i when half i - 3's R is
    // done, a tile's Q when the last R of the tile before is
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_last();
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmQ)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
      int half = 0, q_loads = 0;
      bool ok = true;
      while (ok && walk.next()) {
        if (walk.s.fresh) {
          if (half > 0) ok = !*abort_flag && mbar_wait_bounded(k_empty(half - 1), ((half - 1) / 3) & 1, status, DEV_TIMEOUT_ATTN);
          if (!ok) break;
          mbar_arrive_expect_tx(q_full, Q_BYTES);
          for (int ds = 0; ds < DS; ++ds)
            tma_load_3d(smem_addr(q_s + ds * Q_SLICE), &tmQ, 64 * ds, walk.s.g * a.G, walk.s.row0, q_full, pol);
          ++q_loads;
        }
        for (int h = 0; h < 2; ++h, ++half) {
          if (half >= 3) ok = !*abort_flag && mbar_wait_bounded(k_empty(half), (half / 3 - 1) & 1, status, DEV_TIMEOUT_ATTN);
          if (!ok) break;
          mbar_arrive_expect_tx(k_full(half), KV_BYTES);
          for (int ds = 0; ds < DS; ++ds)
            tma_load_4d(smem_addr(k_s + half % 3 * KV_BYTES + ds * KV_SLICE), &tmK, 64 * ds, walk.s.g,
                        walk.s.k0() + h * kPairs, walk.s.b, k_full(half), pol);
        }
      }
      if (!ok) *abort_flag = 1;
      // loads still in flight (only after an abort) land before the block exits
      if (q_loads > 0) mbar_wait_bounded(q_full, (q_loads - 1) & 1u, nullptr, 0);
      for (int i = max(half - 3, 0); i < half; ++i) mbar_wait_bounded(k_full(i), (i / 3) & 1, nullptr, 0);
    }
    __syncwarp();
  } else if (warp == 18) {
    // ---- V halves, as soon as the step before's products with that half are done
    const uint64_t pol = l2_policy_evict_last();
    auto load = [&](const Step& st, int h) {
      mbar_arrive_expect_tx(v_full(h), KV_BYTES);
      for (int ds = 0; ds < DS; ++ds)
        tma_load_4d(smem_addr(v_s + h * KV_BYTES + ds * KV_SLICE), &tmV, 64 * ds, st.g, st.k0() + h * kPairs, st.b,
                    v_full(h), pol);
    };
    int in_flight[2] = {0, 0};  // loads of each half so far
    bool have = walk.next();
    Step cur = walk.s;
    if (have && lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
      for (int h = 0; h < 2; ++h) {
        load(cur, h);
        ++in_flight[h];
      }
    }
    for (uint32_t ph = 0; have; ph ^= 1) {
      const int k0 = cur.k0();
      const int end = min(kSplit, cur.len_last() - k0);
      const int h0 = max(a.win.sinks - k0, 0), h1 = min(cur.lo - k0, end);  // hidden keys before the window
      for (int h = 0; h < 2; ++h) {
        if (lane == 0 && !mbar_wait_bounded(v_full(h), ph, status, DEV_TIMEOUT_ATTN)) *abort_flag = 1;
        __syncwarp();
        auto zero = [&](int from, int to) {
          from = max(from - h * kPairs, 0);
          to = min(to - h * kPairs, kPairs);
          for (int idx = lane; idx < (to - from) * DS * 8; idx += 32) {
            const int key = from + idx / (DS * 8), rest = idx % (DS * 8);
            *reinterpret_cast<uint4*>(v_s + h * KV_BYTES + (rest / 8) * KV_SLICE + key * 128 + (rest % 8) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        };
        zero(end, kSplit);
        zero(h0, h1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ready(h));
      }
      have = walk.next();
      cur = walk.s;
      if (have && lane == 0) {
        for (int h = 0; h < 2; ++h) {
          if (*abort_flag || !mbar_wait_bounded(v_empty(h), ph, status, DEV_TIMEOUT_ATTN)) {
            *abort_flag = 1;
            break;
          }
          load(cur, h);
          ++in_flight[h];
        }
      }
      if (__shfl_sync(0xffffffffu, *abort_flag, 0) != 0) break;
    }
    if (lane == 0) {
      for (int h = 0; h < 2; ++h)
        if (in_flight[h] > 0) mbar_wait_bounded(v_full(h), (in_flight[h] - 1) & 1u, nullptr, 0);
    }
    __syncwarp();
  } else if (warp == 16) {
    // ---- MMA issue
    if (lane == 0) {
      constexpr uint32_t idesc_r = tc_idesc(128, 0);
      constexpr uint32_t idesc_o = tc_idesc(D, 1);
      // base descriptors; an operand at byte offset b from a base adds b / 16 to
      // the start-address field (shared addresses stay below 256 KB, so the field
      // never carries into the next)
      const uint64_t qd = desc_k_sw128(smem_addr(q_s)), kd = desc_k_sw128(smem_addr(k_s));
      const uint64_t vd = desc_mn_sw128(smem_addr(v_s), KV_SLICE);
      const uint32_t o_col = tmem + 384;
      bool ok = true;
      int half = 0, q_uses = 0;  // halves of R so far
      auto wait = [&](uint32_t b, uint32_t parity) {
        if (!mbar_try_wait(b, parity) && ok) ok = mbar_wait_bounded(b, parity, status, DEV_TIMEOUT_ATTN);
      };
      auto scores = [&](bool new_q) {
        if (new_q) wait(q_full, q_uses++ & 1);
        wait(k_full(half), (half / 3) & 1);
        if (!ok) return;
        const uint64_t k = kd + static_cast<uint64_t>((half % 3 * KV_BYTES) >> 4);
#pragma unroll
        for (int ds = 0; ds < DS; ++ds)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + static_cast<uint32_t>(128 * (half % 3)), qd + static_cast<uint64_t>((ds * Q_SLICE + kk * 32) >> 4),
                      k + static_cast<uint64_t>((ds * KV_SLICE + kk * 32) >> 4), idesc_r, (ds | kk) != 0 ? 1u : 0u);
        umma_commit(k_empty(half));
        ++half;
      };
      // O (+)= P . V over half h of step st, whose P is in buffer (2 st + h) % 3
      auto products = [&](int st, int h) {
        wait(v_ready(h), st & 1);
        // O of the step before is read by threads that have written this half of P
        if (h == 0 && st > 0)
          wait(o_free, (st - 1) & 1);
        else
          wait(p_full(h), st & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t p = tmem + static_cast<uint32_t>(128 * ((2 * st + h) % 3));
        const uint64_t v = vd + static_cast<uint64_t>((h * KV_BYTES) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t p_hi = p + static_cast<uint32_t>(16 * kk);
          const uint64_t vdesc = v + static_cast<uint64_t>((kk * 2048) >> 4);
          umma_bf16_tmem_a(o_col, p_hi, vdesc, idesc_o, (h | kk) != 0 ? 1u : 0u);
          umma_bf16_tmem_a(o_col, p_hi + 8, vdesc, idesc_o, 1u);
        }
        umma_commit(v_empty(h));
      };
      bool more = walk.next();
      if (more) {
        scores(true);
        scores(false);
        if (ok) umma_commit(s_full);
      }
      for (int st = 0; ok && (more || st > 0); ++st) {
        const bool last = !(more = more && walk.next());
        if (!last) scores(walk.s.fresh);
        products(st, 0);
        if (!last) {
          scores(false);
          if (ok) umma_commit(s_full);
        }
        products(st, 1);
        if (ok) umma_commit(o_full);
        if (last) break;
      }
      if (!ok) *abort_flag = 1;
      umma_commit(done_bar);
      mbar_wait_bounded(done_bar, 0, status, DEV_TIMEOUT_ATTN);
    }
    __syncwarp();
  } else {
    // ---- four threads per (row, head) pair
    const int quad = warp & 3, quarter = warp >> 2;      // lanes 32 quad ..; groups quarter, quarter + 4; columns D/4 quarter ..
    const int pr = quad * 32 + lane;                     // pair = TMEM lane
    const int r = pr / a.G, head = pr % a.G;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float c2 = a.c2;
    float o_acc[DQ];
    float m_acc, l_acc;
    bool ok = true;
    // the barrier of the quadrant's four warps, which share their pairs, returning
    // whether `v` holds for any of its threads
    auto quad_sync_or = [&](bool v) {
      uint32_t res;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
          "bar.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(res)
          : "r"(static_cast<uint32_t>(v)), "r"(1 + quad)
          : "memory");
      return res != 0;
    };
    auto wait = [&](uint32_t b, uint32_t parity) {
      const bool waited = mbar_wait_bounded(b, parity, status, DEV_TIMEOUT_ATTN);
      if (__any_sync(0xffffffffu, !waited || *abort_flag)) {
        *abort_flag = 1;
        ok = false;
      }
      tc_fence_after();
    };
    auto begin = [&]() {
#pragma unroll
      for (int d = 0; d < DQ; ++d) o_acc[d] = 0.f;
      m_acc = -INFINITY;
      l_acc = 0.f;
    };
    // folds step sf (maximum mf; whether the pair saw a key) into the running state,
    // this thread's columns of O, once its products are done; PARTS: stores it as partial `part`
    auto fold = [&](int sf, float mf, bool in, int64_t part, int nrows) {
      wait(o_full, sf & 1);
      uint32_t v[DQ];
      const uint32_t col = lane_base + 384 + static_cast<uint32_t>(quarter * DQ);
      if constexpr (DQ == 32)
        tmem_ld32(col, v);
      else
        tmem_ld16(col, v);
      tc_fence_before();
      mbar_arrive(o_free);
      if (!in || (PARTS && (!ok || r >= nrows))) return;
      if (PARTS) {
        float4* to = reinterpret_cast<float4*>(a.parts) + (part * (D / 4) + quarter * (DQ / 4)) * kPairs + pr;
#pragma unroll
        for (int d = 0; d < DQ; d += 4)
          to[d / 4 * kPairs] = make_float4(__uint_as_float(v[d]), __uint_as_float(v[d + 1]), __uint_as_float(v[d + 2]),
                                           __uint_as_float(v[d + 3]));
        if (quarter != 0) return;
      }
      // l: the eight groups' sums in order
      const float* w = x_w + (sf & 1) * 8 * kPairs + pr;
      float lf = w[0];
#pragma unroll
      for (int q = 1; q < 8; ++q) lf = __fadd_rn(lf, w[q * kPairs]);
      if (PARTS) {
        a.parts_ml[part * kPairs + pr] = make_float2(mf, lf);
        return;
      }
      const float m_new = fmaxf(m_acc, mf);
      const float fa = ex2_approx(__fsub_rn(m_acc, m_new));
      const float fc = ex2_approx(__fsub_rn(mf, m_new));
      l_acc = __fadd_rn(__fmul_rn(l_acc, fa), __fmul_rn(lf, fc));
      m_acc = m_new;
      // single operations: a packed add behind packed products is compiled to a fused
      // one, which rounds once where the merge kernel rounds twice
#pragma unroll
      for (int d = 0; d < DQ; ++d)
        o_acc[d] = __fadd_rn(__fmul_rn(o_acc[d], fa), __fmul_rn(__uint_as_float(v[d]), fc));
    };
    // writes the tile's rows
    auto finish = [&](int row0, int nrows, int g) {
      if (!ok || r >= nrows) return;
      __nv_bfloat16* dst = a.out + (static_cast<int64_t>(row0 + r) * a.Hq + g * a.G + head) * D + quarter * DQ;
#pragma unroll
      for (int d = 0; d < DQ; d += 8) {
        uint4 o;
        o.x = pack_bf16(__fdiv_rn(o_acc[d + 0], l_acc), __fdiv_rn(o_acc[d + 1], l_acc));
        o.y = pack_bf16(__fdiv_rn(o_acc[d + 2], l_acc), __fdiv_rn(o_acc[d + 3], l_acc));
        o.z = pack_bf16(__fdiv_rn(o_acc[d + 4], l_acc), __fdiv_rn(o_acc[d + 5], l_acc));
        o.w = pack_bf16(__fdiv_rn(o_acc[d + 6], l_acc), __fdiv_rn(o_acc[d + 7], l_acc));
        *reinterpret_cast<uint4*>(dst + d) = o;
      }
    };
    begin();
    float m_prev = 0.f;
    bool in_prev = false, left = false;
    int prev_row0 = 0, prev_nrows = 0, prev_g = 0;
    int s = 0;
    for (; walk.next(); ++s) {
      const uint32_t ph = s & 1;
      const int k0 = walk.s.k0();
      const int len = walk.s.len0 + r;
      const int cnt = min(kSplit, len - k0);
      // the pair's first window key and the sinks' end within the split
      const int lo = window_lo(a.win, len) - k0, sink = a.win.sinks - k0;
      // every pair of the tile sees the whole split: no key is masked
      const bool whole = walk.s.len0 - k0 >= kSplit &&
                         (window_lo(a.win, walk.s.len_last()) <= k0 || a.win.sinks >= k0 + kSplit);
      auto sees = [&](int key) { return key < cnt && (key >= lo || key < sink); };
      // the thread's group of half h in tensor memory
      auto col_of = [&](int h) {
        return lane_base + static_cast<uint32_t>(128 * ((2 * s + h) % 3) + 32 * quarter);
      };
      wait(s_full, ph);
      // the raw maximum (exact in any order): this thread's two groups of 32 keys, then the pair's
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        tmem_ld32(col_of(h), v);
        if (whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            mx[0] = fmax3(mx[0], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            mx[1] = fmax3(mx[1], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (sees(32 * (quarter + 4 * h) + e)) mx[e & 1] = fmaxf(mx[e & 1], __uint_as_float(v[e]));
        }
      }
      float* xm = x_max + ph * 4 * kPairs + pr;
      xm[quarter * kPairs] = fmaxf(mx[0], mx[1]);
      // one decision for the quadrant's threads: leave if any of them has given up
      if (quad_sync_or(!ok || *abort_flag)) {
        left = true;
        break;
      }
      const float m = __fmul_rn(fmaxf(fmaxf(xm[0], xm[kPairs]), fmaxf(xm[2 * kPairs], xm[3 * kPairs])), c2);
      const float2 c2x2 = make_float2(c2, c2), neg_m2 = make_float2(-m, -m);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = quarter + 4 * h;  // 32-key group of the split
        float sq[4] = {0.f, 0.f, 0.f, 0.f};
        auto weights = [&](auto masked) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t col = col_of(h) + 16 * half;
            uint32_t v[16], hp[8], lp[8];  // bf16 pairs of the high and the low halves
            tmem_ld16(col, v);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 arg = __ffma2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2x2, neg_m2);
              float2 x = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));
              if (decltype(masked)::value) {
                x.x = sees(32 * c + 16 * half + e) ? x.x : 0.f;
                x.y = sees(32 * c + 16 * half + e + 1) ? x.y : 0.f;
              }
              const __nv_bfloat162 h2 = __float22bfloat162_rn(x);
              const __nv_bfloat162 l2 = __float22bfloat162_rn(less_bf16(x, h2));
              hp[e / 2] = *reinterpret_cast<const uint32_t*>(&h2);
              lp[e / 2] = *reinterpret_cast<const uint32_t*>(&l2);
              // the decode kernel's order: key 8nb + 2tq + e into partial tq in (nb, e) order
              sq[e / 2 % 4] = __fadd_rn(__fadd_rn(sq[e / 2 % 4], x.x), x.y);
            }
            tmem_st8(col, hp);
            tmem_st8(col + 8, lp);
          }
        };
        if (whole)
          weights(std::false_type{});
        else
          weights(std::true_type{});
        x_w[(ph * 8 + c) * kPairs + pr] = __fadd_rn(__fadd_rn(sq[0], sq[1]), __fadd_rn(sq[2], sq[3]));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full(h));
        // step s - 1's sums and maximum were published by this step's barrier
        if (h == 0 && s > 0) {
          fold(s - 1, m_prev, in_prev, walk.at_step - 1, prev_nrows);
          if (!PARTS && walk.s.fresh) {
            finish(prev_row0, prev_nrows, prev_g);
            begin();
          }
        }
      }
      m_prev = m;
      in_prev = cnt > 0 && (lo < kSplit || sink > 0);
      prev_row0 = walk.s.row0;
      prev_nrows = walk.s.nrows;
      prev_g = walk.s.g;
    }
    if (!left && s > 0 && !quad_sync_or(!ok || *abort_flag)) {
      fold(s - 1, m_prev, in_prev, walk.at_step, prev_nrows);
      if (!PARTS) finish(prev_row0, prev_nrows, prev_g);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Folds a tile's partials, left to right, and writes its rows: a thread per pair and
// four columns, whose next four partials are on the way while it folds.
constexpr int kFoldThreads = 256;

template <int D>
__global__ void __launch_bounds__(kFoldThreads) prefill_fold_kernel(const Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, pr = threadIdx.x % kPairs;
  const int col4 = blockIdx.y * (kFoldThreads / kPairs) + threadIdx.x / kPairs;
  int before = 0;  // steps of the tiles before this one
#pragma unroll
  for (int j = 0; j < 2; ++j) before += lane_tile_splits(a, lane + 32 * j, blockIdx.x);
  before = __reduce_add_sync(0xffffffffu, before);
  Step s;
  if (!tile_at(a, blockIdx.x, s)) return;
  const int r = pr / a.G, head = pr % a.G;
  if (r >= s.nrows) return;
  const float4* o = reinterpret_cast<const float4*>(a.parts) + (static_cast<int64_t>(before) * (D / 4) + col4) * kPairs + pr;
  const float2* ml = a.parts_ml + static_cast<int64_t>(before) * kPairs + pr;
  const int len = s.len0 + r, first = window_lo(a.win, len);
  float m_acc = -INFINITY, l_acc = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int CH = 4;
  for (int i0 = 0; i0 < s.ns; i0 += CH) {
    float4 ov[CH];
    float2 mlv[CH];
    bool in[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k0 = s.list.split(i0 + i) * kSplit;
      // the row sees a key of the split
      in[i] = i0 + i < s.ns && k0 < len && (first < k0 + kSplit || a.win.sinks > k0);
      if (in[i]) {
        ov[i] = o[static_cast<int64_t>(i0 + i) * (D / 4) * kPairs];
        mlv[i] = ml[static_cast<int64_t>(i0 + i) * kPairs];
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!in[i]) continue;
      const float m_new = fmaxf(m_acc, mlv[i].x);
      const float fa = ex2_approx(__fsub_rn(m_acc, m_new)), fc = ex2_approx(__fsub_rn(mlv[i].x, m_new));
      l_acc = __fadd_rn(__fmul_rn(l_acc, fa), __fmul_rn(mlv[i].y, fc));
      acc.x = __fadd_rn(__fmul_rn(acc.x, fa), __fmul_rn(ov[i].x, fc));
      acc.y = __fadd_rn(__fmul_rn(acc.y, fa), __fmul_rn(ov[i].y, fc));
      acc.z = __fadd_rn(__fmul_rn(acc.z, fa), __fmul_rn(ov[i].z, fc));
      acc.w = __fadd_rn(__fmul_rn(acc.w, fa), __fmul_rn(ov[i].w, fc));
      m_acc = m_new;
    }
  }
  __nv_bfloat16* dst = a.out + (static_cast<int64_t>(s.row0 + r) * a.Hq + s.g * a.G + head) * D + col4 * 4;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(__fdiv_rn(acc.x, l_acc), __fdiv_rn(acc.y, l_acc)),
                                              pack_bf16(__fdiv_rn(acc.z, l_acc), __fdiv_rn(acc.w, l_acc)));
}

// Steps that the tiles of a call can have in all, or 0 where they stay whole.
int64_t parts_steps(int64_t tiles, int RT, int window, int sinks, int max_kv) {
  const int64_t rows = window > 0 ? static_cast<int64_t>(window) + RT - 1 : 0;  // keys that some row of a tile has in its window
  const int64_t splits = max_visible_splits(static_cast<int>(rows < 0x7FFFFFFF ? rows : 0x7FFFFFFF), sinks, max_kv);
  return tiles > kFewTiles || splits < kFewSplits ? 0 : tiles * splits;
}

int64_t tiles_of(int rows, int RT) { return (static_cast<int64_t>(rows) + RT - 1) / RT; }

constexpr size_t part_bytes(int D) { return static_cast<size_t>(kPairs) * (D * 4 + 8); }

template <int D>
constexpr size_t window_smem_bytes() {
  return 1024 + 6 * static_cast<size_t>(D / 64) * kPairs * 128 +
         (2 * 4 + 2 * 8) * kPairs * 4 + (kBars + 1) * 8 + 16;
}

template <int D>
kinv_status launch_window(const void* q, const void* k_cache, const void* v_cache, int64_t seq_stride,
                          int64_t tok_stride, const Args& a, int64_t steps, cudaStream_t stream) {
  CUtensorMap mq, mk, mv;
  const uint64_t qd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.total_rows)};
  const uint64_t qs[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(a.Hq) * D * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(a.RT)};
  const uint64_t kd[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.max_len),
                          static_cast<uint64_t>(a.B)};
  // one sequence: any sequence stride describes it (the coordinate is 0)
  const int64_t sst = a.B > 1 ? seq_stride : static_cast<int64_t>(a.max_len) * tok_stride;
  const uint64_t ks[3] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(tok_stride) * 2,
                          static_cast<uint64_t>(sst) * 2};
  const uint32_t kb[4] = {64, 1, static_cast<uint32_t>(kPairs), 1};  // half a split
  if (!encode_map(&mq, q, 3, qd, qs, qb) || !encode_map(&mk, k_cache, 4, kd, ks, kb) ||
      !encode_map(&mv, v_cache, 4, kd, ks, kb))
    return KINV_ERR_UNSUPPORTED;
  constexpr size_t smem = window_smem_bytes<D>();
  const int tiles = a.tiles_per_seq * a.Hkv * a.B, sms = sm_count();
  if (a.parts) {
    auto kernel = attn_prefill_window_kernel<D, true>;
    kinv_status st = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
    if (st != KINV_OK) return st;
    st = launch_kernel(kernel, dim3(steps < sms ? static_cast<int>(steps) : sms), dim3(kThreads), smem, stream, 1, mq, mk, mv, a);
    if (st != KINV_OK) return st;
    return launch_kernel(prefill_fold_kernel<D>, dim3(tiles, D / 4 / (kFoldThreads / kPairs)), dim3(kFoldThreads), 0, stream, 1, a);
  }
  auto kernel = attn_prefill_window_kernel<D, false>;
  const kinv_status st = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
  if (st != KINV_OK) return st;
  return launch_kernel(kernel, dim3(tiles < sms ? tiles : sms), dim3(kThreads), smem, stream, 1, mq, mk, mv, a);
}

}  // namespace
}  // namespace kinv

using namespace kinv;

extern "C" kinv_status kinv_attn_prefill_window(const void* q, const void* k_cache, const void* v_cache,
                                                int64_t seq_stride, int64_t tok_stride, const int32_t* q_start,
                                                const int32_t* q_len, const int32_t* q_offset, void* out, int B,
                                                int total_rows, int max_q_len, int max_kv, int Hq, int Hkv, int D,
                                                int split_len, int window, int sinks, float scale, void* workspace,
                                                size_t ws_bytes, kinv_stream stream) {
  if (B < 0 || total_rows < 0 || max_q_len < 0 || max_kv < 0 || window < 0 || sinks < 0) return KINV_ERR_INVALID_ARG;
  if (B == 0 || total_rows == 0 || max_q_len == 0) return KINV_OK;
  if (!q || !k_cache || !v_cache || !out || !q_start || !q_len || !q_offset || max_kv <= 0) return KINV_ERR_INVALID_ARG;
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv) return KINV_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return KINV_ERR_UNSUPPORTED;
  if ((D != 64 && D != 128) || split_len != kSplit) return KINV_ERR_UNSUPPORTED;
  if (tok_stride < static_cast<int64_t>(Hkv) * D || seq_stride < 0 || (B > 1 && seq_stride == 0))
    return KINV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || seq_stride % 8 || tok_stride % 8 ||
      !aligned16(workspace))
    return KINV_ERR_ALIGNMENT;
  Args a{};
  a.q_start = q_start;
  a.q_len = q_len;
  a.q_offset = q_offset;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = G;
  a.RT = kPairs / G;
  // a sequence's rows are rows of the call and keys of the cache: a bound above both
  // leaves no room for more tiles (and max_q_len + RT within 32 bits)
  const int most_rows = std::min({max_q_len, total_rows, max_kv});
  a.tiles_per_seq = static_cast<int>(tiles_of(most_rows, a.RT));
  a.max_len = max_kv;
  a.max_q_len = max_q_len;
  a.total_rows = total_rows;
  a.c2 = base2_factor(scale, D);
  a.win = Window{window, sinks};
  // the tiles are counted in an int
  if (B > 65535 || static_cast<int64_t>(a.tiles_per_seq) * Hkv * B > 0x7F000000) return KINV_ERR_UNSUPPORTED;
  a.status = device_status_word();
  const int64_t steps = parts_steps(static_cast<int64_t>(a.tiles_per_seq) * Hkv * B, a.RT, window, sinks, max_kv);
  if (steps > 0 && workspace && ws_bytes >= steps * part_bytes(D)) {
    a.parts = static_cast<float*>(workspace);
    a.parts_ml = reinterpret_cast<float2*>(a.parts + steps * kPairs * D);
  }
  return D == 128 ? launch_window<128>(q, k_cache, v_cache, seq_stride, tok_stride, a, steps, stream)
                  : launch_window<64>(q, k_cache, v_cache, seq_stride, tok_stride, a, steps, stream);
}

extern "C" size_t kinv_attn_prefill_window_workspace(int B, int max_q_len, int Hq, int Hkv, int D, int max_kv,
                                                     int split_len, int window, int sinks) {
  if (B <= 0 || max_q_len <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || D <= 0 || max_kv <= 0 || window < 0 || sinks < 0 ||
      split_len != kSplit || Hq / Hkv > kPairs)
    return 0;
  const int RT = kPairs / (Hq / Hkv);
  return parts_steps(tiles_of(max_q_len, RT) * Hkv * B, RT, window, sinks, max_kv) * part_bytes(D);
}

size_t kinv::most_parts_bytes(int B, int most_rows, int Hq, int Hkv, int D, int max_kv) {
  if (Hq % Hkv || Hq / Hkv > kPairs) return 0;
  const int RT = kPairs / (Hq / Hkv);
  const int64_t per_seq = tiles_of(most_rows, RT), most = kFewTiles / (static_cast<int64_t>(Hkv) * B);
  return parts_steps((per_seq < most ? per_seq : most) * Hkv * B, RT, 0, 0, max_kv) * part_bytes(D);
}
