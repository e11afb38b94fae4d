// Writing the 8-bit key/value cache (with the rotation of a step's rows, or from
// bf16 keys and values) and reading it back.
#include <cmath>

#include "cache8.cuh"
#include "cache8_read.cuh"
#include "rope.cuh"

namespace kinv {
namespace {

// cos and sin of p * inv_freq as rope_angle() forms them, corrected by what the
// reduced angle loses in fp32 (its low part d: cos - d sin, sin + d cos): a
// rounding that goes the other way moves a key's code by a whole step.
__device__ __forceinline__ void rope_angle_corrected(int p, double inv_freq, float& c, float& s) {
  const double theta = static_cast<double>(p) * inv_freq;
  const double k = rint(theta * 0.15915494309189535);  // 1 / (2 pi)
  double red = fma(-k, 6.283185307179586, theta);
  red = fma(-k, 2.4492935982947064e-16, red);
  const float hi = static_cast<float>(red);
  const float d = static_cast<float>(red - static_cast<double>(hi));
  float c0, s0;
  sincosf(hi, &s0, &c0);
  c = __fmaf_rn(-d, s0, c0);
  s = __fmaf_rn(d, c0, s0);
}

__device__ __forceinline__ uint32_t abs_bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x) & 0x7FFFu; }

// kinv_rope_append's layout of work: a block per row and `heads_per_block` of its
// heads, a warp per head; the first D/2 threads form the row's rotation angles.
// A key or value head's largest magnitude is a warp maximum over bit patterns.
constexpr int kRopeWarps = 8;

template <int D, bool I8>
__global__ void rope_append8_kernel(const __nv_bfloat16* __restrict__ qkv, int64_t ld_qkv,
                                    __nv_bfloat16* __restrict__ q_out, const Cache8View cache,
                                    const int32_t* __restrict__ seq, const int32_t* __restrict__ pos,
                                    const __nv_bfloat16* __restrict__ q_norm,
                                    const __nv_bfloat16* __restrict__ k_norm, float eps, int Hq, int Hkv,
                                    int heads_per_block, const RopeFreqs freqs, int* status) {
  constexpr int HALF = D / 2;
  constexpr int P = D / 64;
  __shared__ float cs[HALF], sn[HALF];
  __shared__ __nv_bfloat16 key_rows[kRopeWarps][D];
  pdl_launch_dependents();
  pdl_wait();
  const int r = blockIdx.x;
  const int p = pos[r], s = seq[r];
  if (p < 0 || p >= cache.slots || s < 0 || s >= cache.B) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && status) atomicExch(status, DEV_CACHE8_BAD_RANGE);
    return;
  }
  for (int i = threadIdx.x; i < HALF; i += blockDim.x) rope_angle_corrected(p, freqs.inv_freq[i], cs[i], sn[i]);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const __nv_bfloat16* row = qkv + r * ld_qkv;
  const int64_t tok = s * cache.seq_stride + p * cache.tok_stride;
  const int heads = Hq + 2 * Hkv;
  const int h_end = min(heads, (static_cast<int>(blockIdx.y) + 1) * heads_per_block);
  for (int h = blockIdx.y * heads_per_block + warp; h < h_end; h += nwarps) {
    const __nv_bfloat16* src = row + h * D;
    if (h >= Hq + Hkv) {  // value head
      const int g = h - Hq - Hkv;
      uint32_t w[P];
      if (P == 2) {
        const uint2 v = reinterpret_cast<const uint2*>(src)[lane];
        w[0] = v.x;
        w[P - 1] = v.y;
      } else {
        w[0] = reinterpret_cast<const uint32_t*>(src)[lane];
      }
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < P; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
      const int E = scale_exponent<I8>(__reduce_max_sync(0xffffffffu, m));
      const float inv = encode_factor(E);
      uint32_t code = encode2<I8>(bf16_lo(w[0]), bf16_hi(w[0]), inv);
      unsigned char* dst = cache.v + tok + g * D;
      if (P == 2) {
        code |= encode2<I8>(bf16_lo(w[P - 1]), bf16_hi(w[P - 1]), inv) << 16;
        reinterpret_cast<uint32_t*>(dst)[lane] = code;
      } else {
        reinterpret_cast<uint16_t*>(dst)[lane] = static_cast<uint16_t>(code);
      }
      if (lane == 0) cache.ve[s * cache.eseq_stride + g * cache.ehead_stride + p] = static_cast<int8_t>(E);
      continue;
    }
    float a[P], b[P], c[P], sv[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      a[j] = __bfloat162float(src[lane * P + j]);
      b[j] = __bfloat162float(src[HALF + lane * P + j]);
      c[j] = cs[lane * P + j];
      sv[j] = sn[lane * P + j];
    }
    if (h < Hq) {
      rope_norm_rotate<D>(a, b, c, sv, q_norm, eps, lane, q_out + (static_cast<int64_t>(r) * Hq + h) * D);
      continue;
    }
    // the rotated key by way of shared memory, each lane its own values
    __nv_bfloat16* turned = key_rows[warp];
    rope_norm_rotate<D>(a, b, c, sv, k_norm, eps, lane, turned);
    __nv_bfloat16 lo[P], hi[P];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      lo[j] = turned[lane * P + j];
      hi[j] = turned[HALF + lane * P + j];
      m = max(m, max(abs_bits(lo[j]), abs_bits(hi[j])));
    }
    const int E = scale_exponent<I8>(__reduce_max_sync(0xffffffffu, m));
    const float inv = encode_factor(E);
    const int g = h - Hq;
    unsigned char* dst = cache.k + tok + g * D;
    if (P == 2) {
      const uint32_t x = encode2<I8>(__bfloat162float(lo[0]), __bfloat162float(lo[P - 1]), inv);
      const uint32_t y = encode2<I8>(__bfloat162float(hi[0]), __bfloat162float(hi[P - 1]), inv);
      reinterpret_cast<uint16_t*>(dst)[lane] = static_cast<uint16_t>(x);
      reinterpret_cast<uint16_t*>(dst + HALF)[lane] = static_cast<uint16_t>(y);
    } else {
      const uint32_t x = encode2<I8>(__bfloat162float(lo[0]), __bfloat162float(hi[0]), inv);
      dst[lane] = static_cast<unsigned char>(x);
      dst[HALF + lane] = static_cast<unsigned char>(x >> 8);
    }
    if (lane == 0) cache.ke[s * cache.eseq_stride + g * cache.ehead_stride + p] = static_cast<int8_t>(E);
  }
}

// bf16 keys (z = 0) or values (z = 1) of `tokens` tokens of one sequence: a group
// of D / 8 lanes per (token, head), 16 bytes a lane, four vectors a lane ahead.
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
  constexpr int AHEAD = 4;
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
      const float inv = encode_factor(E);
      if (tok[j] < 0) continue;
      uint2 c;
      c.x = encode2<I8>(bf16_lo(x[j].x), bf16_hi(x[j].x), inv) | (encode2<I8>(bf16_lo(x[j].y), bf16_hi(x[j].y), inv) << 16);
      c.y = encode2<I8>(bf16_lo(x[j].z), bf16_hi(x[j].z), inv) | (encode2<I8>(bf16_lo(x[j].w), bf16_hi(x[j].w), inv) << 16);
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
const RopeFreqs& rope_freqs(float base, int D) {
  static thread_local RopeFreqs freqs;
  static thread_local float of_base = 0.f;
  static thread_local int of_dim = 0;
  if (base != of_base || D != of_dim) {
    for (int i = 0; i < D / 2; ++i) freqs.inv_freq[i] = std::pow(static_cast<double>(base), -2.0 * i / D);
    of_base = base;
    of_dim = D;
  }
  return freqs;
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
  if (!aligned16(qkv) || !aligned16(q_out) || ld_qkv % 8) return KINV_ERR_ALIGNMENT;
  const RopeFreqs& freqs = rope_freqs(rope_base, D);
  const int heads = Hq + 2 * Hkv;
  const int hpb = rows >= 512 ? heads : 8;  // as kinv_rope_append
  const dim3 grid(rows, (heads + hpb - 1) / hpb);
  auto run = [&](auto kernel) {
    return launch_kernel(kernel, grid, dim3(32 * kRopeWarps), 0, stream, 1, static_cast<const __nv_bfloat16*>(qkv), ld_qkv,
                         static_cast<__nv_bfloat16*>(q_out), view, seq, pos,
                         static_cast<const __nv_bfloat16*>(q_norm), static_cast<const __nv_bfloat16*>(k_norm), eps,
                         Hq, Hkv, hpb, freqs, device_status_word());
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
  p.max_len = max_len;
  p.Hkv = Hkv;
  p.status = device_status_word();
  p.tokens = tokens_per_block(B, max_len, Hkv, D);
  const dim3 grid((max_len + p.tokens - 1) / p.tokens, B, 2);
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
  p.max_len = max_len;
  p.Hkv = Hkv;
  p.status = device_status_word();
  return launch_cache8_read(p, cache->dtype == KINV_I8, B, D, stream);
}
