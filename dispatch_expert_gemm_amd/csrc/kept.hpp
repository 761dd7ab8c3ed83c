// Values kept in 8 bits (rule at moe_swiglu_checkpoint_fwd in moe.h): a block of 32
// consecutive columns of a row has one bf16 scale s = bf16(amax / 127) and int8 codes
// rint(v * fp32(1 / s)).  Four neighbouring lanes hold a block, eight columns each;
// its amax comes from two lane permutations on the values' bits, where an infinity
// and a NaN order above every number.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kKeptCols = 32;  // columns of a block

// Scale bits and the multiplier of a block from the largest bf16 magnitude's bits.
// The product with fp32(1/127) rounds to the same bf16 as amax / 127: that quotient
// of an 8-bit mantissa by 127 is over 2^-17 of its value away from any midpoint of
// two bf16 numbers.  One Newton step makes v_rcp_f32's result the rounded
// reciprocal (tested for every scale).
__device__ __forceinline__ uint32_t kept_scale(uint32_t amax16, float& inv) {
  const uint32_t s = pk_bf16(__fmul_rn(bf2f(amax16), 1.0f / 127.0f), 0.f);
  const float sf = bf2f(s), r = __builtin_amdgcn_rcpf(sf);
  const bool some = s >= 0x0080u && amax16 < 0x7f80u;
  inv = some ? __fmaf_rn(__fmaf_rn(-sf, r, 1.0f), r, r) : 0.f;
  return amax16 >= 0x7f80u ? 0x7fc0u : (some ? s : 0u);
}

__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}

// Largest magnitude (bf16 bits) of the 32 values that four neighbouring lanes hold.
__device__ __forceinline__ uint32_t block_amax(const uint4& v) {
  constexpr uint32_t k = 0x7fff7fffu;
  uint32_t m = max16x2(max16x2(v.x & k, v.y & k), max16x2(v.z & k, v.w & k));
  m = max16x2(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));
  m = max16x2(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));
  const uint32_t hi = m >> 16, lo = m & 0xffffu;
  return hi > lo ? hi : lo;
}

// The code of v in the low byte.  |v * inv| <= 127 (1 + 2^-8), so adding 1.5 * 2^23 to
// the rounded product (no contraction: the rule rounds it to fp32 first) leaves rint
// of it, ties to even, in the sum's low bits.
__device__ __forceinline__ uint32_t code(float v, float inv) {
#pragma clang fp contract(off)
  const float p = v * inv;
  return __float_as_uint(p + 12582912.0f);
}

// Four codes in a word.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  const uint32_t lo = __builtin_amdgcn_perm(code(b, inv), code(a, inv), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(code(d, inv), code(c, inv), 0x04000c0cu);
  return lo | hi;
}

__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
  float f[8];
  unpack8(v, f);
  const uint32_t lo = codes4(f[0], f[1], f[2], f[3], inv), hi = codes4(f[4], f[5], f[6], f[7], inv);
  // inv 0: zeros, or an infinity or a NaN among them (whose products are none)
  return inv == 0.f ? make_uint2(0u, 0u) : make_uint2(lo, hi);
}

// Eight kept values: code * s, exact in fp32.
__device__ __forceinline__ void kept8(const uint2& q, float s, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __fmul_rn((float)(int8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3))), s);
}

}  // namespace moe
