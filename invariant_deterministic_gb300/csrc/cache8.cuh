// The 8-bit key/value cache: codes, scales and their conversions.
//
// A (token, kv head) holds D codes and one exponent E (int8), for its key and
// for its value vector each; element d stands for code[d] * 2^E.  With amax the
// largest magnitude of the D bf16 values,
//   e4m3:  E = the smallest e with amax <= 448 * 2^e, in [-100, 119]
//   int8:  E = the smallest e with amax <= 127 * 2^e, in [-100, 121]
//   code   = x * 2^-E rounded to the nearest code, ties to even, saturating
// and E = -128 marks a vector that held an infinity or a NaN: all of it stands
// for NaN.  The scale is a power of two so that code * 2^E is a bf16 number
// exactly (e4m3 has 4 significant bits, int8 7): reading back loses nothing, and
// an attention kernel that scales before or after its products gets the bits of
// attention over the cache read back.  It costs e4m3 no accuracy and int8 at
// most one bit.  The upper bounds keep 448 * 2^119 and 127 * 2^121 finite in
// bf16.  One token per scale, because a block of several would have to be
// rounded again when a louder token joins it, and what a row sees would then
// depend on which later tokens the cache already holds.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace kinv {

constexpr int DEV_CACHE8_BAD_RANGE = dev_code(10, KINV_ERR_INVALID_ARG);

constexpr int kExpNaN = -128;
constexpr int kExpMin = -100;

template <bool I8>
__host__ __device__ constexpr int exp_max() {
  return I8 ? 121 : 119;
}

struct Cache8View {
  unsigned char* k;
  unsigned char* v;
  int8_t* ke;
  int8_t* ve;
  int64_t seq_stride, tok_stride;    // codes (bytes)
  int64_t eseq_stride, ehead_stride; // exponents
  int B, slots;
};

// E from the largest bf16 magnitude's bits (sign cleared): amax = (1 + m/128) *
// 2^(e - 127); 448 = (1 + 96/128) 2^8, 127 = (1 + 126/128) 2^6.
template <bool I8>
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 7), m = static_cast<int>(amax_bits & 0x7F);
  if (e == 255) return kExpNaN;
  const int E = I8 ? e - 133 + (m > 126) : e - 135 + (m > 96);
  return min(max(E, kExpMin), exp_max<I8>());
}

// 2^E as fp32; NaN for the mark.
__device__ __forceinline__ float exponent_factor(int E) {
  return E == kExpNaN ? __int_as_float(0x7FFFFFFF) : __int_as_float(max(E + 127, 0) << 23);
}

// The codes of four bf16 values (two words of pairs) with exponent E, the first in the
// low byte.  int8: x * 2^-E + 1.5 * 2^23 is rounded to an integer whose low byte is the
// code; only a vector with the largest E can reach 128.
template <bool I8>
__device__ __forceinline__ uint32_t encode4(uint32_t w0, uint32_t w1, int E) {
  if (E == kExpNaN) return 0u;
  const float inv = __int_as_float((127 - E) << 23);
  const float2 inv2 = make_float2(inv, inv);
  const float2 x = make_float2(bf16_lo(w0), bf16_hi(w0)), y = make_float2(bf16_lo(w1), bf16_hi(w1));
  if (I8) {
    const float2 half = make_float2(12582912.f, 12582912.f);
    float2 a = __ffma2_rn(x, inv2, half), b = __ffma2_rn(y, inv2, half);
    if (E == exp_max<true>()) {
      a = make_float2(fminf(fmaxf(a.x, 12582912.f - 127.f), 12582912.f + 127.f), fminf(fmaxf(a.y, 12582912.f - 127.f), 12582912.f + 127.f));
      b = make_float2(fminf(fmaxf(b.x, 12582912.f - 127.f), 12582912.f + 127.f), fminf(fmaxf(b.y, 12582912.f - 127.f), 12582912.f + 127.f));
    }
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
  }
  return __nv_cvt_float2_to_fp8x2(__fmul2_rn(x, inv2), __NV_SATFINITE, __NV_E4M3) |
         (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(__fmul2_rn(y, inv2), __NV_SATFINITE, __NV_E4M3)) << 16);
}

// Four codes (a word) as two bf16 pairs: bytes 0 and 2, and bytes 1 and 3.
// e4m3 s eeee mmm becomes the bf16 bits s 0000eeee mmm0000, which is the code's
// value * 2^-120 for normal and subnormal codes alike (codes 7F and FF, which no
// writer here makes, read as +-480 * 2^-120: every byte is a finite number).
// int8: the bf16 number with bits 0x00uu is uu * 2^-133, subnormal or not; with the
// sign bit flipped the byte is v + 128, and uu * 2^-6 - 2 is v * 2^-6 exactly (one
// product and sum a pair beside the masks: 64 sequences over 4,096 int8 keys 98 us,
// 111 with three integer steps and a difference).
// The exponent that is missing.
template <bool I8>
__host__ __device__ constexpr int expand_exp() {
  return I8 ? 6 : 120;
}

template <bool I8>
__device__ __forceinline__ void expand4(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (I8) {
    const uint32_t e = (w ^ 0x80808080u) & 0x00FF00FFu, o = ((w >> 8) ^ 0x00800080u) & 0x00FF00FFu;
    const __nv_bfloat162 up = __bfloat162bfloat162(__ushort_as_bfloat16(0x7F00));   // 2^127
    const __nv_bfloat162 off = __bfloat162bfloat162(__ushort_as_bfloat16(0xC000));  // -2
    const __nv_bfloat162 x = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&e), up, off);
    const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&o), up, off);
    even = *reinterpret_cast<const uint32_t*>(&x);
    odd = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    even = ((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u);
    odd = ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u);
  }
}

// Four codes as two f16 pairs in their order, exactly (every e4m3 number and
// every int8 is an f16 number; codes 7F and FF become NaN, which nothing reads).
// int8: with the sign bit flipped the byte is v + 128, and 1024 + (v + 128) is an
// f16 number whose low byte it is.
template <bool I8>
__device__ __forceinline__ void expand4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (I8) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// The bf16 pair (code 2j, code 2j + 1) of a word's codes, j = 0, 1, times 2^E.
template <bool I8>
__device__ __forceinline__ uint2 decode4(uint32_t w, float factor) {
  uint32_t even, odd;
  expand4<I8>(w, even, odd);
  const float lift = I8 ? 0x1p6f : 0x1p120f;
  const float e0 = __fmul_rn(__fmul_rn(bf16_lo(even), lift), factor), e1 = __fmul_rn(__fmul_rn(bf16_hi(even), lift), factor);
  const float o0 = __fmul_rn(__fmul_rn(bf16_lo(odd), lift), factor), o1 = __fmul_rn(__fmul_rn(bf16_hi(odd), lift), factor);
  return make_uint2(pack_bf16(e0, o0), pack_bf16(e1, o1));
}

// The host's checks of a kinv_cache8 for heads of D values.
inline kinv_status check_cache8(const kinv_cache8* c, int Hkv, int D, Cache8View* view) {
  if (!c || !c->k || !c->v || !c->k_exp || !c->v_exp || c->B < 0 || c->slots < 0 || Hkv <= 0) return KINV_ERR_INVALID_ARG;
  if (c->dtype != KINV_E4M3 && c->dtype != KINV_I8) return KINV_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return KINV_ERR_UNSUPPORTED;
  if (c->tok_stride < static_cast<int64_t>(Hkv) * D || c->seq_stride < 0 || c->exp_seq_stride < 0 ||
      (Hkv > 1 && c->exp_head_stride < c->slots))
    return KINV_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || c->seq_stride % 16 || c->tok_stride % 16) return KINV_ERR_ALIGNMENT;
  view->k = static_cast<unsigned char*>(c->k);
  view->v = static_cast<unsigned char*>(c->v);
  view->ke = c->k_exp;
  view->ve = c->v_exp;
  view->seq_stride = c->seq_stride;
  view->tok_stride = c->tok_stride;
  view->eseq_stride = c->exp_seq_stride;
  view->ehead_stride = c->exp_head_stride;
  view->B = c->B;
  view->slots = c->slots;
  return KINV_OK;
}

}  // namespace kinv
