// Reading the 8-bit cache back into bf16: for kinv_cache8_read, and for the keys
// and values that a prompt chunk's rows see.
#pragma once

#include "cache8.cuh"
#include "window.cuh"

namespace kinv {

constexpr int kReadThreads = 256;

// Tokens of one block of the kernels that write the cache or read it back: 32
// (a sector of exponents a head) where that leaves four blocks to an SM, else
// fewer, down to about one vector a lane: few tokens cost a load's latency for
// each round of a block (500 tokens of 8 heads of 128: 17.4 us by 32, 3.7 by 2).
inline int tokens_per_block(int B, int max_len, int Hkv, int D) {
  int tokens = 32;
  const int64_t want = 4 * static_cast<int64_t>(sm_count());
  while (tokens > 1 && 2 * static_cast<int64_t>(B) * ((max_len + tokens - 1) / tokens) < want &&
         tokens * Hkv * (D / 8) > kReadThreads)
    tokens /= 2;
  return tokens;
}

struct ReadParams {
  Cache8View cache;
  __nv_bfloat16* k;   // token i of sequence b, head g at b*seq_stride + i*tok_stride + g*D
  __nv_bfloat16* v;
  int64_t seq_stride, tok_stride;
  const int32_t* start;  // token i is slot start[b] + i, i < len[b] ...
  const int32_t* len;
  const int32_t* q_start;  // ... or, with these, slot i < q_start[b] + q_len[b] where a row of the chunk sees it
  const int32_t* q_len;
  int max_len, max_q_len, Hkv, tokens;
  Window win;
  int* status;
};

// Keys (z = 0) or values (z = 1) of `tokens` tokens of one sequence, D / 16
// lanes per (token, head): 16 codes in, 32 bytes out a lane, two vectors ahead.
// Writing and reading back 8 x 32,768 tokens of 8 heads of 128 take 547 us, 5.9 TB/s
// (four ahead 561, half as many codes a lane 569).
template <int D, bool I8>
__global__ void __launch_bounds__(kReadThreads) cache8_read_kernel(const ReadParams p) {
  constexpr int L = D / 16;
  constexpr int PER = kReadThreads / L;
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y;
  int start = 0, len, lo = 0;
  if (p.q_start) {
    // the attention kernel behind this one reports sequences outside the bounds
    const int s0 = p.q_start[b], n = p.q_len[b];
    if (n <= 0 || n > p.max_q_len || s0 < 0 || s0 > p.max_len - n) return;
    len = s0 + n;
    lo = window_lo(p.win, s0 + 1);
  } else {
    start = p.start[b];
    len = p.len[b];
    if (start < 0 || len < 0 || len > p.max_len || start > p.cache.slots - len) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && p.status) atomicExch(p.status, DEV_CACHE8_BAD_RANGE);
      return;
    }
  }
  const int i0 = blockIdx.x * p.tokens;
  const int n = min(p.tokens, len - i0);
  if (n <= 0 || (i0 >= p.win.sinks && i0 + n <= lo)) return;
  const bool values = blockIdx.z != 0;
  const unsigned char* src = (values ? p.cache.v : p.cache.k) + b * p.cache.seq_stride;
  const int8_t* exps = (values ? p.cache.ve : p.cache.ke) + b * p.cache.eseq_stride + start + i0;
  __nv_bfloat16* dst = (values ? p.v : p.k) + b * p.seq_stride;
  const int sub = threadIdx.x % L;
  src += (start + i0) * p.cache.tok_stride + sub * 16;
  dst += i0 * p.tok_stride + sub * 16;
  const int total = n * p.Hkv;
  constexpr int AHEAD = 2;
  for (int at = threadIdx.x / L; at < total; at += PER * AHEAD) {
    uint4 c[AHEAD];
    int e[AHEAD], tok[AHEAD], head[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int vec = at + j * PER;
      tok[j] = vec < total ? vec / p.Hkv : -1;
      head[j] = vec - tok[j] * p.Hkv;
      if (tok[j] >= 0) {
        c[j] = __ldcs(reinterpret_cast<const uint4*>(src + tok[j] * p.cache.tok_stride + head[j] * D));
        e[j] = exps[head[j] * p.cache.ehead_stride + tok[j]];
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (tok[j] < 0) continue;
      const float f = exponent_factor(e[j]);
      const uint2 x0 = decode4<I8>(c[j].x, f), x1 = decode4<I8>(c[j].y, f), x2 = decode4<I8>(c[j].z, f),
                  x3 = decode4<I8>(c[j].w, f);
      uint4* to = reinterpret_cast<uint4*>(dst + tok[j] * p.tok_stride + head[j] * D);
      to[0] = make_uint4(x0.x, x0.y, x1.x, x1.y);
      to[1] = make_uint4(x2.x, x2.y, x3.x, x3.y);
    }
  }
}

inline kinv_status launch_cache8_read(ReadParams p, bool i8, int B, int D, cudaStream_t stream) {
  p.tokens = tokens_per_block(B, p.max_len, p.Hkv, D);
  const dim3 grid((p.max_len + p.tokens - 1) / p.tokens, B, 2);
  auto run = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kReadThreads), 0, stream, 1, p); };
  if (D == 128) return i8 ? run(cache8_read_kernel<128, true>) : run(cache8_read_kernel<128, false>);
  return i8 ? run(cache8_read_kernel<64, true>) : run(cache8_read_kernel<64, false>);
}

}  // namespace kinv
