// Writing the 8-bit key/value cache (with the rotation of a step's rows, or from
// bf16 keys and values) and reading it back.
#include <cmath>

#include "cache8.cuh"
#include "cache8_read.cuh"

namespace kinv {
namespace {

// Frequencies base^(-2i/D) in turns, formed in fp64 and held as 64-bit fractions (the
// last bit 0): p times one of them, modulo 2^64, is the angle's fraction of a turn to
// p 2^-63 of a turn beside p times the fp64 frequency's own error.
struct RopeTurns {
  uint64_t turn[64];
};

// A number as the sum of two floats, the second below half a step of the first.
struct Two {
  float h, l;
};

// a + b exactly, |a| >= |b| or a = 0.
__device__ __forceinline__ Two fast_sum(float a, float b) {
  const float h = __fadd_rn(a, b);
  return {h, __fadd_rn(__fsub_rn(a, h), b)};
}

__device__ __forceinline__ Two product_of(float a, float b) {
  const float h = __fmul_rn(a, b);
  return {h, __fmaf_rn(a, b, -h)};
}

// cos and sin of the angle of position p, rounded to fp32 from 2^-27: integers instead of
// kinv_rope_append's fp64 (this GPU does two fp64 operations a cycle and SM) down to an
// eighth of a turn, then the Taylor series with their first terms in two floats (a
// rounding that goes the other way moves a key's code by a whole step).
__device__ __forceinline__ void rope_angle_turns(int p, uint64_t turn, float& c, float& s) {
  const uint64_t x = static_cast<uint64_t>(static_cast<uint32_t>(p)) * turn;  // fraction of a turn * 2^64
  const uint32_t quarter = static_cast<uint32_t>((x + (1ull << 61)) >> 62);
  const int64_t y = static_cast<int64_t>(x - (static_cast<uint64_t>(quarter) << 62));
  // y = (h + l) 2^38, h exact as a float
  const float h = static_cast<float>(static_cast<int32_t>(y >> 38));
  const float l = __fmul_rn(static_cast<float>(static_cast<uint32_t>(y >> 6)), 0x1p-32f);
  constexpr double kTurn = 6.283185307179586476925 * 0x1p-26;  // radians of a unit of h
  constexpr float kHi = static_cast<float>(kTurn), kLo = static_cast<float>(kTurn - static_cast<double>(kHi));
  const Two a0 = product_of(h, kHi);
  const Two a = fast_sum(a0.h, __fadd_rn(a0.l, __fmaf_rn(h, kLo, __fmul_rn(l, kHi))));
  Two z = product_of(a.h, a.h);
  z.l = __fmaf_rn(__fmul_rn(2.f, a.h), a.l, z.l);
  // cos = 1 - z / 2 + z^2 (1/4! - z/6! + z^2/8! - z^3/10!)
  float t = __fmaf_rn(z.h, -1.f / 3628800.f, 1.f / 40320.f);
  t = __fmaf_rn(z.h, t, -1.f / 720.f);
  t = __fmaf_rn(z.h, t, 1.f / 24.f);
  const Two c0 = fast_sum(1.f, __fmul_rn(-0.5f, z.h));
  const Two cc = fast_sum(c0.h, __fadd_rn(c0.l, __fmaf_rn(__fmul_rn(z.h, z.h), t, __fmul_rn(-0.5f, z.l))));
  // sin = a - a z / 3! + a z^2 (1/5! - z/7! + z^2/9! - z^3/11!)
  t = __fmaf_rn(z.h, -1.f / 39916800.f, 1.f / 362880.f);
  t = __fmaf_rn(z.h, t, -1.f / 5040.f);
  t = __fmaf_rn(z.h, t, 1.f / 120.f);
  Two q = product_of(a.h, z.h);
  q.l = __fadd_rn(q.l, __fmaf_rn(a.h, z.l, __fmul_rn(a.l, z.h)));
  constexpr float kSixth = 1.f / 6.f, kSixthLo = static_cast<float>(1.0 / 6.0 - static_cast<double>(kSixth));
  const Two w = product_of(q.h, kSixth);
  const float wl = __fadd_rn(w.l, __fmaf_rn(q.h, kSixthLo, __fmul_rn(q.l, kSixth)));
  const Two s0 = fast_sum(a.h, -w.h);
  const Two ss = fast_sum(s0.h, __fadd_rn(s0.l, __fadd_rn(__fsub_rn(a.l, wl), __fmul_rn(__fmul_rn(q.h, z.h), t))));
  const bool swap = quarter & 1, minus_c = (quarter + 1) & 2, minus_s = quarter & 2;
  c = swap ? ss.h : cc.h;
  s = swap ? cc.h : ss.h;
  if (minus_c) c = -c;
  if (minus_s) s = -s;
}

// D / 16 lanes hold a head, each lane eight rotation pairs (i, i + D/2) in two 16-byte
// loads, so a warp takes four heads of 128 (eight of 64) at a time.  A block has one
// row, or as many as make one wave of blocks, at most sixteen; its threads form the
// angles together beside the first loads, and each warp asks for its next heads before
// it works on the last.  What bounds many rows: about 16 us for each 4,096 (5.7 TB/s),
// and about 4 us that do not depend on them, a block's positions, angles and barrier in
// the only wave there is (4,096 rows of the 8B shape 20.6 us, 4,864 22.6, 9,728 41.3,
// 16,384 68.7).  To keep the instructions below that (68 % of the issue slots at 4,096
// rows) fp32 products go in pairs, gains and angles stand in shared memory in the order
// of the lanes, and nothing is converted by the slow unit that a sum can round.  Before
// those steps 4,096 rows took 26.7 us with four rows a block whatever the number of
// blocks, 41 with a row a block, 37 with a warp per head, a pair of values a lane and
// angles in fp64, as kinv_rope_append has it.
constexpr int kAppendRows = 16;
constexpr int kAppendBlocks = 4;  // of 256 threads on an SM

struct Append8Params {
  const __nv_bfloat16* qkv;
  int64_t ld_qkv;
  __nv_bfloat16* q_out;
  Cache8View cache;
  const int32_t* seq;
  const int32_t* pos;
  const __nv_bfloat16* q_norm;
  const __nv_bfloat16* k_norm;
  float eps;
  int rows, rows_per_block, Hq, Hkv;
  RopeTurns turns;
  int* status;
};

template <int D, bool I8>
__global__ void __launch_bounds__(512, 2) rope_append8_kernel(const __grid_constant__ Append8Params a) {
  constexpr int HALF = D / 2;
  constexpr int L = D / 16;   // lanes of a head
  constexpr int HPW = 32 / L; // heads of a warp
  __shared__ __align__(16) float cs[kAppendRows][HALF], sn[kAppendRows][HALF], minus_sn[kAppendRows][HALF];
  __shared__ __align__(16) float gains[2][D];  // of queries, of keys
  __shared__ int place[kAppendRows][2];  // of each row: sequence (-1: outside the cache), position
  // where number i of a half stands: the lanes' first four beside each other, then their others
  auto slot = [](int i) { return (i >> 2 & 1) * (HALF / 2) + (i >> 3) * 4 + (i & 3); };
  pdl_launch_dependents();
  pdl_wait();
  const int r0 = blockIdx.x * a.rows_per_block, n = min(a.rows_per_block, a.rows - r0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L;
  const int heads = a.Hq + 2 * a.Hkv;
  const int groups = (heads + HPW - 1) / HPW;  // of a row, a warp's work at a time
  const __nv_bfloat16* base = a.qkv + r0 * a.ld_qkv + sub * 8;
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  int row = warp / groups, group = warp - row * groups;
  auto load = [&]() {
    const int h = group * HPW + lane / L;
    if (row < n && h < heads) {
      lo = *reinterpret_cast<const uint4*>(base + row * a.ld_qkv + h * D);
      hi = *reinterpret_cast<const uint4*>(base + row * a.ld_qkv + h * D + HALF);
    }
  };
  load();
  if (threadIdx.x < n) {
    const int p = a.pos[r0 + threadIdx.x], s = a.seq[r0 + threadIdx.x];
    const bool fits = p >= 0 && p < a.cache.slots && s >= 0 && s < a.cache.B;
    place[threadIdx.x][0] = fits ? s : -1;
    place[threadIdx.x][1] = p;
    if (!fits && a.status) atomicExch(a.status, DEV_CACHE8_BAD_RANGE);
  }
  const int at = threadIdx.x % HALF, step = blockDim.x / HALF;  // this thread's frequency, and rows at a time
  if (threadIdx.x < step * HALF) {
    const uint64_t turn = a.turns.turn[at];
    for (int i = threadIdx.x / HALF; i < n; i += step) {
      float c, sv;
      rope_angle_turns(a.pos[r0 + i], turn, c, sv);
      cs[i][slot(at)] = c;
      sn[i][slot(at)] = sv;
      minus_sn[i][slot(at)] = -sv;
    }
  }
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    const int to = i / HALF * HALF + slot(i % HALF);
    if (a.q_norm) gains[0][to] = __bfloat162float(a.q_norm[i]);
    if (a.k_norm) gains[1][to] = __bfloat162float(a.k_norm[i]);
  }
  __syncthreads();
  // whole warps, so that every lane takes part in the shuffles
  while (row < n) {
    const int h = group * HPW + lane / L, first = group * HPW, now = row;
    const int s = place[now][0], p = place[now][1];
    const int64_t r = r0 + now;
    const bool live = h < heads && s >= 0, value = h >= a.Hq + a.Hkv;
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};  // the head's bf16 pairs: low half, high half
    for (group += blockDim.x >> 5; group >= groups; group -= groups) ++row;
    load();
    const bool normed = live && !value && (h < a.Hq ? a.q_norm : a.k_norm) != nullptr;
    float2 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = make_float2(bf16_lo(w[j]), bf16_hi(w[j]));
    if (__any_sync(0xffffffffu, normed)) {
      float2 acc2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
      for (int j = 1; j < 8; ++j) acc2 = __ffma2_rn(x[j], x[j], acc2);
      float acc = __fadd_rn(acc2.x, acc2.y);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, o));
      if (normed) {
        const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(acc, 1.f / D), a.eps)));
        const float* g = gains[h < a.Hq ? 0 : 1] + sub * 4;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 gv = *reinterpret_cast<const float4*>(g + j / 2 * (HALF / 2));
          x[j] = __fmul2_rn(__fmul2_rn(x[j], make_float2(inv, inv)), make_float2(gv.x, gv.y));
          x[j + 1] = __fmul2_rn(__fmul2_rn(x[j + 1], make_float2(inv, inv)), make_float2(gv.z, gv.w));
        }
      }
    }
    if (!value) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float4 c = *reinterpret_cast<const float4*>(&cs[now][sub * 4 + j / 2 * (HALF / 2)]),
                     sv = *reinterpret_cast<const float4*>(&sn[now][sub * 4 + j / 2 * (HALF / 2)]),
                     ns = *reinterpret_cast<const float4*>(&minus_sn[now][sub * 4 + j / 2 * (HALF / 2)]);
        const float2 cc[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
        const float2 ss[2] = {make_float2(sv.x, sv.y), make_float2(sv.z, sv.w)};
        const float2 nn[2] = {make_float2(ns.x, ns.y), make_float2(ns.z, ns.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 u = x[j + e], v = x[4 + j + e];
          x[j + e] = __ffma2_rn(u, cc[e], __fmul2_rn(v, nn[e]));
          x[4 + j + e] = __ffma2_rn(v, cc[e], __fmul2_rn(u, ss[e]));
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = pack_bf16(x[j].x, x[j].y);
    }
    if (live && h < a.Hq) {
      __nv_bfloat16* dst = a.q_out + (r * a.Hq + h) * D + sub * 8;
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(dst + HALF) = make_uint4(w[4], w[5], w[6], w[7]);
    }
    if (first + HPW <= a.Hq) continue;  // query heads only
    // the largest magnitude by bit patterns
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!live || h < a.Hq) continue;
    const int E = scale_exponent<I8>(max(m & 0xFFFFu, m >> 16));
    uint32_t code[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) code[j] = encode4<I8>(w[2 * j], w[2 * j + 1], E);
    const int g = value ? h - a.Hq - a.Hkv : h - a.Hq;
    unsigned char* dst =
        (value ? a.cache.v : a.cache.k) + s * a.cache.seq_stride + p * a.cache.tok_stride + g * D + sub * 8;
    *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
    *reinterpret_cast<uint2*>(dst + HALF) = make_uint2(code[2], code[3]);
    if (sub == 0)
      (value ? a.cache.ve : a.cache.ke)[s * a.cache.eseq_stride + g * a.cache.ehead_stride + p] = static_cast<int8_t>(E);
  }
}

// bf16 keys (z = 0) or values (z = 1) of `tokens` tokens of one sequence: a group
// of D / 8 lanes per (token, head), 16 bytes a lane, two vectors a lane ahead.
// The exponents of the block go out together, one run of bytes a head.
constexpr int kWriteThreads = 256;

struct WriteParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t seq_stride, tok_stride;
  const int32_t* start;
  const int32_t* len;
  int max_len, Hkv, tokens;
  Cache8View cache;
  int* status;
};

template <int D, bool I8>
__global__ void __launch_bounds__(kWriteThreads) cache8_write_kernel(const WriteParams p) {
  constexpr int L = D / 8;                      // lanes of a vector
  constexpr int PER = kWriteThreads / L;        // vectors at a time
  constexpr int AHEAD = 2;
  extern __shared__ int8_t exps[];              // [Hkv][tokens]
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y;
  const int start = p.start[b], len = p.len[b];
  if (start < 0 || len < 0 || len > p.max_len || start > p.cache.slots - len) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.status) atomicExch(p.status, DEV_CACHE8_BAD_RANGE);
    return;
  }
  const int i0 = blockIdx.x * p.tokens;
  const int n = min(p.tokens, len - i0);
  if (n <= 0) return;
  const bool values = blockIdx.z != 0;
  const int sub = threadIdx.x % L;
  const __nv_bfloat16* src = (values ? p.v : p.k) + b * p.seq_stride + i0 * p.tok_stride + sub * 8;
  unsigned char* dst =
      (values ? p.cache.v : p.cache.k) + b * p.cache.seq_stride + (start + i0) * p.cache.tok_stride + sub * 8;
  const int total = n * p.Hkv;
  // whole rounds, so that every lane takes part in the shuffles
  for (int at = 0; at < total; at += PER * AHEAD) {
    uint4 x[AHEAD];
    int tok[AHEAD], head[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int vec = at + j * PER + static_cast<int>(threadIdx.x) / L;
      tok[j] = vec < total ? vec / p.Hkv : -1;
      head[j] = vec - tok[j] * p.Hkv;
      x[j] = make_uint4(0, 0, 0, 0);
      if (tok[j] >= 0) x[j] = __ldcs(reinterpret_cast<const uint4*>(src + tok[j] * p.tok_stride + head[j] * D));
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      uint32_t m = __vmaxu2(__vmaxu2(x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu),
                            __vmaxu2(x[j].z & 0x7FFF7FFFu, x[j].w & 0x7FFF7FFFu));
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int E = scale_exponent<I8>(max(m & 0xFFFFu, m >> 16));
      if (tok[j] < 0) continue;
      const uint2 c = make_uint2(encode4<I8>(x[j].x, x[j].y, E), encode4<I8>(x[j].z, x[j].w, E));
      *reinterpret_cast<uint2*>(dst + tok[j] * p.cache.tok_stride + head[j] * D) = c;
      if (sub == 0) exps[head[j] * p.tokens + tok[j]] = static_cast<int8_t>(E);
    }
  }
  __syncthreads();
  int8_t* e = (values ? p.cache.ve : p.cache.ke) + b * p.cache.eseq_stride + start + i0;
  for (int idx = threadIdx.x; idx < p.tokens * p.Hkv; idx += kWriteThreads) {
    const int g = idx / p.tokens, i = idx % p.tokens;
    if (i < n) e[g * p.cache.ehead_stride + i] = exps[idx];
  }
}

// The last table a thread asked for: 64 powers are 4 us of a call.
const RopeTurns& rope_turns(float base, int D) {
  static thread_local RopeTurns turns;
  static thread_local float of_base = 0.f;
  static thread_local int of_dim = 0;
  if (base != of_base || D != of_dim) {
    for (int i = 0; i < D / 2; ++i) {
      // turns a position, less whole ones (a base below 1 has frequencies above 1)
      const double f = std::pow(static_cast<double>(base), -2.0 * i / D) * 0.15915494309189533577;  // 1 / (2 pi)
      turns.turn[i] = static_cast<uint64_t>(std::ldexp(f - std::floor(f), 63)) << 1;
    }
    of_base = base;
    of_dim = D;
  }
  return turns;
}

constexpr int kMaxKvHeads = 1024;  // the write kernel's exponents: 32 bytes a head in shared memory

}  // namespace
}  // namespace kinv

using namespace kinv;

extern "C" kinv_status kinv_rope_append8(const void* qkv, int64_t ld_qkv, void* q_out, const kinv_cache8* cache,
                                         const int32_t* seq, const int32_t* pos, const void* q_norm,
                                         const void* k_norm, float eps, int rows, int Hq, int Hkv, int D,
                                         float rope_base, kinv_stream stream) {
  if (rows < 0 || Hq <= 0 || Hkv <= 0 || !(rope_base > 0.f) || !(eps >= 0.f)) return KINV_ERR_INVALID_ARG;
  Cache8View view;
  const kinv_status st = check_cache8(cache, Hkv, D, &view);
  if (st != KINV_OK) return st;
  if (cache->B > 1 && (cache->seq_stride == 0 || cache->exp_seq_stride == 0)) return KINV_ERR_INVALID_ARG;
  if (rows == 0) return KINV_OK;
  if (!qkv || !q_out || !seq || !pos || ld_qkv < static_cast<int64_t>(Hq + 2 * Hkv) * D) return KINV_ERR_INVALID_ARG;
  if (!aligned16(qkv) || !aligned16(q_out) || ld_qkv % 8 || (q_norm && !aligned16(q_norm)) ||
      (k_norm && !aligned16(k_norm)))
    return KINV_ERR_ALIGNMENT;
  Append8Params p{static_cast<const __nv_bfloat16*>(qkv), ld_qkv, static_cast<__nv_bfloat16*>(q_out), view, seq, pos,
                  static_cast<const __nv_bfloat16*>(q_norm), static_cast<const __nv_bfloat16*>(k_norm), eps, rows, 1, Hq, Hkv,
                  rope_turns(rope_base, D), device_status_word()};
  const int per_warp = 32 / (D / 16);
  int warps = (Hq + 2 * Hkv + per_warp - 1) / per_warp;
  const int resident = kAppendBlocks * sm_count();
  if (rows > resident) {
    const int64_t a_wave = static_cast<int64_t>(resident) * kAppendRows, waves = (rows + a_wave - 1) / a_wave;
    p.rows_per_block = static_cast<int>((rows + resident * waves - 1) / (resident * waves));
    warps = warps * p.rows_per_block < 8 ? warps * p.rows_per_block : 8;
  }
  if (warps < D / 64) warps = D / 64;  // a thread for each of a row's angles
  auto run = [&](auto kernel) {
    return launch_kernel(kernel, dim3((rows + p.rows_per_block - 1) / p.rows_per_block), dim3(32 * (warps < 16 ? warps : 16)), 0,
                         stream, 1, p);
  };
  const bool i8 = cache->dtype == KINV_I8;
  if (D == 128) return i8 ? run(rope_append8_kernel<128, true>) : run(rope_append8_kernel<128, false>);
  return i8 ? run(rope_append8_kernel<64, true>) : run(rope_append8_kernel<64, false>);
}

namespace kinv {
namespace {
kinv_status check_ranges(const void* k, const void* v, int64_t seq_stride, int64_t tok_stride,
                         const kinv_cache8* cache, const int32_t* start, const int32_t* len, int B, int max_len,
                         int Hkv, int D, Cache8View* view) {
  if (B < 0 || max_len < 0) return KINV_ERR_INVALID_ARG;
  const kinv_status st = check_cache8(cache, Hkv, D, view);
  if (st != KINV_OK) return st;
  if (B > cache->B) return KINV_ERR_INVALID_ARG;
  if (B == 0 || max_len == 0) return KINV_OK;
  if (!k || !v || !start || !len || tok_stride < static_cast<int64_t>(Hkv) * D || seq_stride < 0)
    return KINV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || seq_stride % 8 || tok_stride % 8) return KINV_ERR_ALIGNMENT;
  if (B > 65535 || Hkv > kMaxKvHeads) return KINV_ERR_UNSUPPORTED;
  return KINV_OK;
}

// No sequence of more tokens than the cache has slots fits, so a bound above them asks
// for no more blocks (one at least, which reports what does not fit).
int most_tokens(int max_len, const kinv_cache8& cache) {
  const int slots = cache.slots > 0 ? cache.slots : 1;
  return max_len < slots ? max_len : slots;
}
}  // namespace
}  // namespace kinv

extern "C" kinv_status kinv_cache8_write(const void* k, const void* v, int64_t seq_stride, int64_t tok_stride,
                                         const kinv_cache8* cache, const int32_t* start, const int32_t* len, int B,
                                         int max_len, int Hkv, int D, kinv_stream stream) {
  WriteParams p{};
  const kinv_status st = check_ranges(k, v, seq_stride, tok_stride, cache, start, len, B, max_len, Hkv, D, &p.cache);
  if (st != KINV_OK || B == 0 || max_len == 0) return st;
  if (B > 1 && (cache->seq_stride == 0 || cache->exp_seq_stride == 0)) return KINV_ERR_INVALID_ARG;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.seq_stride = seq_stride;
  p.tok_stride = tok_stride;
  p.start = start;
  p.len = len;
  p.max_len = most_tokens(max_len, *cache);
  p.Hkv = Hkv;
  p.status = device_status_word();
  p.tokens = tokens_per_block(B, p.max_len, Hkv, D);
  const dim3 grid((p.max_len + p.tokens - 1) / p.tokens, B, 2);
  const size_t smem = static_cast<size_t>(Hkv) * p.tokens;
  auto run = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kWriteThreads), smem, stream, 1, p); };
  const bool i8 = cache->dtype == KINV_I8;
  if (D == 128) return i8 ? run(cache8_write_kernel<128, true>) : run(cache8_write_kernel<128, false>);
  return i8 ? run(cache8_write_kernel<64, true>) : run(cache8_write_kernel<64, false>);
}

extern "C" kinv_status kinv_cache8_read(const kinv_cache8* cache, const int32_t* start, const int32_t* len, void* k,
                                        void* v, int64_t seq_stride, int64_t tok_stride, int B, int max_len, int Hkv,
                                        int D, kinv_stream stream) {
  ReadParams p{};
  const kinv_status st = check_ranges(k, v, seq_stride, tok_stride, cache, start, len, B, max_len, Hkv, D, &p.cache);
  if (st != KINV_OK || B == 0 || max_len == 0) return st;
  if (B > 1 && seq_stride == 0) return KINV_ERR_INVALID_ARG;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.seq_stride = seq_stride;
  p.tok_stride = tok_stride;
  p.start = start;
  p.len = len;
  p.max_len = most_tokens(max_len, *cache);
  p.Hkv = Hkv;
  p.status = device_status_word();
  return launch_cache8_read(p, cache->dtype == KINV_I8, B, D, stream);
}
