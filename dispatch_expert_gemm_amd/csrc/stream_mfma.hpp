// Products of a few activation rows with weights that are read once: the wave
// level of the few-token layer and of the int8 matrix product's small-M form.
//
// A wave multiplies 16 weight rows (output columns) with up to 16 * RT
// activation rows over a range of the contraction, in steps of 64 bytes per row
// (32 bf16 or 64 int8 values): v_mfma_f32_16x16x32_bf16 or
// v_mfma_i32_16x16x64_i8, the weights the first operand.  Lane l holds 16 bytes
// of weight row l % 16 and of activation row l % 16, both at chunk l / 16 of the
// step, so operands go from memory to the matrix cores in the layout they are
// stored in, with no LDS and no shuffles; the result's lane l holds columns
// 4 (l / 16) .. + 3 of activation row l % 16.  A product's column depends on its
// own activation row alone, so a lane without a row of its own may read any
// valid row: its results are dropped.
#pragma once

#include "common.hpp"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

template <bool I8>
struct MfmaAcc {
  typedef f32x4 type;
};
template <>
struct MfmaAcc<true> {
  typedef i32x4_t type;
};

template <bool I8>
__device__ __forceinline__ typename MfmaAcc<I8>::type mfma16(const i32x4_t& w, const i32x4_t& x,
                                                             typename MfmaAcc<I8>::type c) {
  if constexpr (I8)
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0,
                                                   0, 0);
}

constexpr int kStepBytes = 64;  // bytes of every row in one step

// Steps of a row of `bytes` bytes (a multiple of 16; the last step may be partial).
__host__ __device__ inline int stream_steps(int64_t bytes) { return (int)((bytes + kStepBytes - 1) / kStepBytes); }

// A value that every lane of the wave holds, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ i32x4_t ld16(const char* base, uint32_t off) {
  return *reinterpret_cast<const i32x4_t*>(base + (size_t)off);
}

// acc[n][r] += (16 weight rows n) x (16 activation rows r) over steps [s0, s1) of
// rows of `bytes` bytes.  A lane's chunk of step s of weight rows n is at
// w[n] + 64 s + woff[n], of activation rows r, plane p, at x[p] + 64 s + xoff[r]
// (PX planes, each multiplied with the same weights); w, x, s0 and s1 are the
// same in every lane, so they stay in scalar registers.  U steps' loads are
// issued before their products.
template <bool I8, int NW, int RT, int PX, int U>
__device__ __forceinline__ void stream_mfma(const char* const (&w)[NW], const uint32_t (&woff)[NW],
                                            const char* const (&x)[PX], const uint32_t (&xoff)[RT], int64_t bytes,
                                            int s0, int s1, typename MfmaAcc<I8>::type (&acc)[NW][RT]) {
  const int full = (int)(bytes / kStepBytes);
  const int e = s1 < full ? s1 : full;
  int s = s0;
  for (; s + U <= e; s += U) {
    i32x4_t wv[U][NW], xv[U][PX][RT];
    const int64_t o = (int64_t)s * kStepBytes;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int n = 0; n < NW; ++n) wv[u][n] = ld16(w[n] + o + u * kStepBytes, woff[n]);
#pragma unroll
      for (int p = 0; p < PX; ++p)
#pragma unroll
        for (int r = 0; r < RT; ++r) xv[u][p][r] = ld16(x[p] + o + u * kStepBytes, xoff[r]);
    }
    __builtin_amdgcn_sched_barrier(0);  // every load of the U steps before the first product
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < NW; ++n)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int p = 0; p < PX; ++p) acc[n][r] = mfma16<I8>(wv[u][n], xv[u][p][r], acc[n][r]);
  }
  for (; s < s1; ++s) {
    const int64_t o = (int64_t)s * kStepBytes;
    // past the row's end (only in the last, partial step) both operands are zero
    const bool in = o + 16 * (int)((threadIdx.x % kWave) / 16) < bytes;
    const i32x4_t z = {0, 0, 0, 0};
    i32x4_t wv[NW], xv[PX][RT];
#pragma unroll
    for (int n = 0; n < NW; ++n) wv[n] = in ? ld16(w[n] + o, woff[n]) : z;
#pragma unroll
    for (int p = 0; p < PX; ++p)
#pragma unroll
      for (int r = 0; r < RT; ++r) xv[p][r] = in ? ld16(x[p] + o, xoff[r]) : z;
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int p = 0; p < PX; ++p) acc[n][r] = mfma16<I8>(wv[n], xv[p][r], acc[n][r]);
  }
}

// amax over the workgroup's values (red: one float per wave; every thread gets it).
template <int WAVES>
__device__ __forceinline__ float block_max(float m, float* red) {
  m = wave_max64(m);
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = m;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) r = fmaxf(r, red[i]);
  __syncthreads();
  return r;
}

// The int8 rule's multiplier and scale of a row of maximum magnitude m.  The
// multiplier stays finite, so a zero in a row of tiny values (m < 2^-121) keeps
// code 0.
__device__ __forceinline__ void int8_scale(float m, float& inv, float& scale) {
  inv = m > 0.f ? fminf(__fdiv_rn(127.0f, m), 3.402823466e38f) : 0.f;
  scale = m > 0.f ? __fdiv_rn(m, 127.0f) : 1.0f;
}

// One row of n values (n a multiple of 8) to int8 by a workgroup of 64 * WAVES
// threads: codes clamp(rint(v * (127 / amax)), -127, 127), scale amax / 127 (an
// all-zero row: codes 0, scale 1).  get8(i, f) gives values 8 i .. 8 i + 7; it is
// called in an amax pass and again for the codes, which go to put2(i, codes).
template <int WAVES, class Get, class Put>
__device__ __forceinline__ float quant_row_int8(int64_t n, float* red, Get get8, Put put2) {
  float m = 0.f;
  for (int64_t i = threadIdx.x; i < n / 8; i += WAVES * kWave) {
    float f[8];
    get8(i, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(f[q]));
  }
  float inv, scale;
  int8_scale(block_max<WAVES>(m, red), inv, scale);
  for (int64_t i = threadIdx.x; i < n / 8; i += WAVES * kWave) {
    float f[8];
    get8(i, f);
    put2(i, make_uint2(i8x4(f[0], f[1], f[2], f[3], inv), i8x4(f[4], f[5], f[6], f[7], inv)));
  }
  return scale;
}

}  // namespace moe
