// Products of a few activation rows with weights that are read once: the wave
// level of the few-token layer and of the int8 matrix product's small-M form.
//
// A wave multiplies NW groups of 16 weight rows (output columns) with up to 16 RT
// activation rows over a range of the contraction, in steps of 128 bytes per row
// (64 bf16 or 128 int8 values): v_mfma_f32_16x16x32_bf16 or v_mfma_i32_16x16x64_i8,
// the weights the first operand.  Both operands go from memory straight into a
// small LDS ring of the wave's own, eight rows of 128 bytes by each load, so every
// request is a whole cache line (rows of 64 bytes spread over the lanes as the
// matrix cores take them reached 37 against 94 bytes per ns and CU), and no
// barrier is needed: the wave waits for its own loads by count.  Fragments then
// are read as 16 bytes of row l % 16, chunk 4 kk + l / 16; the result's lane l
// holds columns 4 (l / 16) .. + 3 of activation row l % 16.  A product's column
// depends on its own activation row alone, so what a lane without a row holds
// does not matter.
#pragma once

#include <atomic>

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

constexpr int kStepBytes = 128;  // bytes of every row in one step

// Steps of a row of `bytes` bytes (a multiple of 16; the last step may be partial).
__host__ __device__ inline int stream_steps(int64_t bytes) { return (int)((bytes + kStepBytes - 1) / kStepBytes); }

// A value that every lane of the wave holds, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// s_waitcnt immediate: at most n vector memory operations outstanding (LDS reads:
// none)
constexpr int vm_wait(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// Raw buffer over `bytes` bytes (at most 2^31) at p, in scalar registers: accesses
// past it read zeros.
__device__ __forceinline__ i32x4_t buffer_of(const void* p, int64_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return i32x4_t{uniform((int)(uint32_t)v), uniform((int)(uint32_t)(v >> 32) & 0xffff),
                 uniform((int)(bytes < 0 ? 0 : bytes)), 0x00020000};
}
constexpr uint32_t kPastBuffer = 0x80000000u;

// One 16-byte-per-lane load from buffer offset vo (per lane) + so into LDS at `lds`
// (+ 16 lane).  It has no register result; the pipelines wait for it by count.
__device__ __forceinline__ void load_lds(const i32x4_t& r, const char* lds, uint32_t vo, uint32_t so) {
  const uint32_t m0 = (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)(lds));
  asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" : : "v"(vo), "s"(r), "s"(so), "{m0}"(m0));
}

// Chunk position of chunk c (16 bytes) of row r in LDS rows of 128 bytes: the 16 rows
// that one read phase takes lie in 16 different slots of a 256-byte window.
__device__ __forceinline__ int swizzle(int r, int c) { return c ^ ((r >> 1) & 7); }

// Lane l's row (of 16, its half j) and chunk byte in a row group's loads.
__device__ __forceinline__ int stream_row(int j) { return 8 * j + (threadIdx.x % kWave) / 8; }
__device__ __forceinline__ uint32_t stream_chunk(int j) {
  return 16 * swizzle(stream_row(j), threadIdx.x % 8);
}

// Bytes of one ring slot; a wave's ring is D of them.  RT = 0: the weights alone.
template <int NW, int RT, int PX>
constexpr int kSlot = (NW + PX * RT) * 2048;

// Rows of int8 codes that a workgroup holds in LDS whole: bytes of one (a multiple of
// 128, so the last step reads zeros past the end, and 64 more, so that neighbouring
// rows lie in different banks).
__host__ __device__ inline int held_pitch(int64_t len) { return (int)((len + 127) / 128 * 128 + 64); }

// fp32 rows of n values (a multiple of 32) lie in two planes, blocks of 32 values in
// turn: plane p's row holds blocks p, p + 2, ..., so that a step of 64 values is 128
// bytes of either plane.  Bytes of a plane's row, and the place of value i of row r.
__host__ __device__ inline int64_t plane_pitch(int64_t n) { return (n + 63) / 64 * 128; }
__device__ __forceinline__ float* plane_at(float* const (&plane)[2], int64_t n, int64_t r, int64_t i) {
  return plane[i / 32 % 2] + r * (plane_pitch(n) / 4) + i / 64 * 32 + i % 32;
}

// Eight fp32 values as three bf16 parts whose sum is the value, every bit of it: each
// part takes the 8 leading bits of what is left (24 in all).  An infinity is its high
// part alone; in a NaN every part is one.
__device__ __forceinline__ void bf16_parts(const i32x4_t (&v)[2], i32x4_t (&part)[3]) {
  float f[8], r[8], peak = 0.f;
  uint32_t hi[8], mid[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    f[q] = __int_as_float(v[q / 4][q % 4]);
    hi[q] = __float_as_uint(f[q]) & 0xffff0000u;
    r[q] = f[q] - __uint_as_float(hi[q]);
    peak = fmaxf(peak, fabsf(f[q]));
  }
  if (__builtin_expect(__ballot(peak == __builtin_inff()) != 0, 0)) {
#pragma unroll
    for (int q = 0; q < 8; ++q) r[q] = fabsf(f[q]) == __builtin_inff() ? 0.f : r[q];
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    mid[q] = __float_as_uint(r[q]) & 0xffff0000u;
    r[q] -= __uint_as_float(mid[q]);
  }
#pragma unroll
  for (int q = 0; q < 8; q += 2) {
    auto upper = [&](uint32_t a, uint32_t b) { return (int)__builtin_amdgcn_perm(b, a, 0x07060302u); };
    part[0][q / 2] = upper(hi[q], hi[q + 1]);
    part[1][q / 2] = upper(mid[q], mid[q + 1]);
    part[2][q / 2] = upper(__float_as_uint(r[q]), __float_as_uint(r[q + 1]));
  }
}

// acc[n][r] += (weight rows of group n) x (activation rows of tile r) over steps
// [s0, s1) of weight rows of `bytes` bytes.  w[n]: a buffer of group n's rows (its end
// also ends the valid rows); x[p]: a buffer of plane p's activation rows, xoff[r][j] the
// byte offset of row stream_row(j) of tile r in it, kPastBuffer for none (XI = 1: tiles
// of at most 8 rows).  PX = 1: rows like the weights'; PX = 2: fp32 rows in two planes,
// for bf16 weights: their three parts are multiplied with the same weight registers.
// (The rows as two bf16 parts, 16 bits of each value, read the same bytes: a layer of 64
// tokens on 8 experts of 4096 x 14336 515 against 505 us here with top 2, 705 against 715 with
// top 8; of 1536 x 512 with top 8, where the parts' formation shows, 31.6 against 36.7.  The
// parts as three planes, written once: 541 against 498, 762 against 716, 34.7 against 36.6.)
// ring: D slots of LDS.  w, x, s0 and s1 are the same in every lane.
template <bool I8, int NW, int RT, int PX, int XI, int D>
__device__ __forceinline__ void stream_mfma(const i32x4_t (&w)[NW], const i32x4_t (&x)[PX],
                                            const uint32_t (&xoff)[RT][XI], int64_t bytes, int s0, int s1, char* ring,
                                            typename MfmaAcc<I8>::type (&acc)[NW][RT]) {
  constexpr int I = 2 * NW + PX * RT * XI;  // loads of one slot
  const int lane = threadIdx.x % kWave;
  const uint32_t nb = (uint32_t)bytes;
  uint32_t woff[2], xo[RT][XI];
#pragma unroll
  for (int j = 0; j < 2; ++j) woff[j] = stream_row(j) * nb + stream_chunk(j);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < XI; ++j) xo[r][j] = xoff[r][j] == kPastBuffer ? kPastBuffer : xoff[r][j] + stream_chunk(j);
  auto issue = [&](char* slot, int s) {
    const uint32_t o = (uint32_t)s * kStepBytes;
    uint32_t wo[2] = {woff[0], woff[1]}, xs[PX][RT][XI];
#pragma unroll
    for (int p = 0; p < PX; ++p)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < XI; ++j) xs[p][r][j] = xo[r][j];
    if (o + kStepBytes > nb) {
      // the last, partial step: chunks past the row's end read zeros (PX = 2: half a
      // step of the weights is a block of the first plane, and none of the second)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (o + stream_chunk(j) >= nb) wo[j] = kPastBuffer;
#pragma unroll
      for (int j = 0; j < XI; ++j)
        if (PX == 2 || o + stream_chunk(j) >= nb)
#pragma unroll
          for (int r = 0; r < RT; ++r) xs[PX - 1][r][j] = kPastBuffer;
    }
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) load_lds(w[n], slot + n * 2048 + j * 1024, wo[j], o);
#pragma unroll
    for (int p = 0; p < PX; ++p)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < XI; ++j) load_lds(x[p], slot + (NW + p * RT + r) * 2048 + j * 1024, xs[p][r][j], o);
  };
  const int n = s1 - s0;
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < n) issue(ring + d * kSlot<NW, RT, PX>, s0 + d);
  int at[2];  // this lane's fragments in a row group
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) at[kk] = (lane % 16) * 128 + 16 * swizzle(lane % 16, 4 * kk + lane / 16);
  int atf[2];  // and in a plane's: eight fp32 values
#pragma unroll
  for (int h = 0; h < 2; ++h) atf[h] = (lane % 16) * 128 + 16 * swizzle(lane % 16, 2 * (lane / 16) + h);
  auto step = [&](char* slot, int i) {
    // the slot's loads have arrived: later ones may be outstanding
    if (i + D - 1 < n) __builtin_amdgcn_s_waitcnt(vm_wait(I * (D - 1)));
    else __builtin_amdgcn_s_waitcnt(vm_wait(0));
    asm volatile("" ::: "memory");
    i32x4_t wv[2][NW], xv[2][RT][PX];  // (PX = 2: block kk's eight values in two halves)
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int g = 0; g < NW; ++g) wv[kk][g] = *reinterpret_cast<const i32x4_t*>(slot + g * 2048 + at[kk]);
#pragma unroll
      for (int p = 0; p < PX; ++p)
#pragma unroll
        for (int r = 0; r < RT; ++r)
          xv[kk][r][p] = *reinterpret_cast<const i32x4_t*>(
              PX == 1 ? slot + (NW + r) * 2048 + at[kk] : slot + (NW + kk * RT + r) * 2048 + atf[p]);
    }
    // every fragment is in registers: the slot takes the loads of a later step
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (i + D < n) issue(slot, s0 + i + D);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if constexpr (PX == 1) {
#pragma unroll
          for (int g = 0; g < NW; ++g) acc[g][r] = mfma16<I8>(wv[kk][g], xv[kk][r][0], acc[g][r]);
        } else {
          static_assert(!I8, "fp32 rows go with bf16 weights");
          i32x4_t part[3];
          bf16_parts(xv[kk][r], part);
#pragma unroll
          for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int g = 0; g < NW; ++g) acc[g][r] = mfma16<I8>(wv[kk][g], part[p], acc[g][r]);
        }
      }
  };
  for (int i = 0; i < n; i += D) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (i + d < n) step(ring + d * kSlot<NW, RT, PX>, i + d);
  }
}

// The same for one tile of int8 rows that the workgroup holds in LDS: `held` is this
// lane's row (any row, for a lane without one), chunk l / 16.
template <int NW, int D, class Between>
__device__ __forceinline__ void stream_held(const i32x4_t (&w)[NW], const char* held, int64_t bytes, int s0, int s1,
                                            char* ring, i32x4_t (&acc)[NW], Between between) {
  constexpr int I = 2 * NW;
  const int lane = threadIdx.x % kWave;
  const uint32_t nb = (uint32_t)bytes;
  uint32_t woff[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) woff[j] = stream_row(j) * nb + stream_chunk(j);
  auto issue = [&](char* slot, int s) {
    const uint32_t o = (uint32_t)s * kStepBytes;
    uint32_t wo[2] = {woff[0], woff[1]};
    if (o + kStepBytes > nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (o + stream_chunk(j) >= nb) wo[j] = kPastBuffer;
    }
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) load_lds(w[n], slot + n * 2048 + j * 1024, wo[j], o);
  };
  const int n = s1 - s0;
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < n) issue(ring + d * kSlot<NW, 0, 0>, s0 + d);
  between();
  int at[2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) at[kk] = (lane % 16) * 128 + 16 * swizzle(lane % 16, 4 * kk + lane / 16);
  auto step = [&](char* slot, int i) {
    if (i + D - 1 < n) __builtin_amdgcn_s_waitcnt(vm_wait(I * (D - 1)));
    else __builtin_amdgcn_s_waitcnt(vm_wait(0));
    asm volatile("" ::: "memory");
    i32x4_t wv[2][NW], xv[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int g = 0; g < NW; ++g) wv[kk][g] = *reinterpret_cast<const i32x4_t*>(slot + g * 2048 + at[kk]);
      xv[kk] = *reinterpret_cast<const i32x4_t*>(held + (s0 + i) * kStepBytes + 64 * kk);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (i + D < n) issue(slot, s0 + i + D);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int g = 0; g < NW; ++g) acc[g] = mfma16<true>(wv[kk][g], xv[kk], acc[g]);
  };
  for (int i = 0; i < n; i += D) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (i + d < n) step(ring + d * kSlot<NW, 0, 0>, i + d);
  }
}

// A row's largest magnitude is found on the bits of |v|, which order as the values do,
// with infinity and then NaN above them: a row that holds a NaN gets a scale of NaN and
// does not pass for a finite one.
__device__ __forceinline__ void peak_of(uint32_t& m, float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  m = b > m ? b : m;
}
__device__ __forceinline__ uint32_t wave_peak(uint32_t m) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint32_t v = (uint32_t)__shfl_xor((int)m, o, kWave);
    m = v > m ? v : m;
  }
  return m;
}
// The largest of the waves' peaks.
template <int WAVES>
__device__ __forceinline__ float peak_in(const uint32_t* red) {
  uint32_t m = red[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) m = red[i] > m ? red[i] : m;
  return __uint_as_float(m);
}

// The int8 rule's multiplier and scale of a row of maximum magnitude m.  127 / m is
// 127 times the rounded reciprocal, as a program of tensor operations forms it: a value
// on a border between two codes (half the maximum is one: 63.5) then goes the way it
// goes there.  The multiplier stays finite, so a zero in a row of tiny values
// (m < 2^-121) keeps code 0; infinity and NaN go into the scale.
__device__ __forceinline__ void int8_scale(float m, float& inv, float& scale) {
  inv = m == 0.f ? 0.f : fminf(__fmul_rn(127.0f, __fdiv_rn(1.0f, m)), 3.402823466e38f);
  scale = m == 0.f ? 1.0f : __fdiv_rn(m, 127.0f);
}

// ROWS rows of n values (n a multiple of 8, at most 8 PER values for every thread) to
// int8 by a workgroup of 64 WAVES threads: codes clamp(rint(v * (127 / amax)), -127,
// 127), scale amax / 127 (an all-zero row: codes 0, scale 1).  get8(r, i, f) gives values
// 8 i .. 8 i + 7 of row r < rows, put2(r, i, codes) takes them, scale(r, s) the scales.
// red: ROWS * WAVES words of LDS.
template <int WAVES, int ROWS, int PER, class Get, class Put, class Scale>
__device__ __forceinline__ void quant_rows_int8(int rows, int64_t n, uint32_t* red, Get get8, Put put2, Scale scale) {
  float f[ROWS][PER][8];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int i = threadIdx.x + p * WAVES * kWave;
      if (r < rows && i < n / 8) {
        get8(r, i, f[r][p]);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[r][p][q] = 0.f;
      }
    }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p)
#pragma unroll
      for (int q = 0; q < 8; ++q) peak_of(m, f[r][p][q]);
    m = wave_peak(m);
    if (threadIdx.x % kWave == 0) red[r * WAVES + threadIdx.x / kWave] = m;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (r >= rows) break;
    float inv, s;
    int8_scale(peak_in<WAVES>(red + r * WAVES), inv, s);
    if (threadIdx.x == 0) scale(r, s);
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int i = threadIdx.x + p * WAVES * kWave;
      const float* v = f[r][p];
      if (i < n / 8) put2(r, i, make_uint2(i8x4(v[0], v[1], v[2], v[3], inv), i8x4(v[4], v[5], v[6], v[7], inv)));
    }
  }
}

// One row of any length: the row in registers if it fits, else read twice.
template <int WAVES, class Get, class Put>
__device__ __forceinline__ float quant_row_int8(int64_t n, uint32_t* red, Get get8, Put put2) {
  float sc = 0.f;
  if (n <= 4 * 8 * WAVES * kWave) {
    quant_rows_int8<WAVES, 1, 4>(
        1, n, red, [&](int, int64_t i, float* f) { get8(i, f); }, [&](int, int64_t i, uint2 c) { put2(i, c); },
        [&](int, float s) { sc = s; });
    return sc;
  }
  uint32_t m = 0;
  for (int64_t i = threadIdx.x; i < n / 8; i += WAVES * kWave) {
    float f[8];
    get8(i, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) peak_of(m, f[q]);
  }
  m = wave_peak(m);
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = m;
  __syncthreads();
  float inv;
  int8_scale(peak_in<WAVES>(red), inv, sc);
  for (int64_t i = threadIdx.x; i < n / 8; i += WAVES * kWave) {
    float f[8];
    get8(i, f);
    put2(i, make_uint2(i8x4(f[0], f[1], f[2], f[3], inv), i8x4(f[4], f[5], f[6], f[7], inv)));
  }
  return sc;
}

// One row of any length by one wave, the values in registers up to 4096 of them.
template <class Get, class Put>
__device__ __forceinline__ float quant_row_int8_wave(int64_t n, Get get8, Put put2) {
  constexpr int PER = 8;
  const int lane = threadIdx.x % kWave;
  const bool held = n <= PER * 8 * kWave;
  float f[PER][8], inv, sc;
  uint32_t m = 0;
  if (held) {
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      if (lane + p * kWave < n / 8) {
        get8(lane + p * kWave, f[p]);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[p][q] = 0.f;
      }
    }
#pragma unroll
    for (int p = 0; p < PER; ++p)
#pragma unroll
      for (int q = 0; q < 8; ++q) peak_of(m, f[p][q]);
  } else {
    for (int64_t i = lane; i < n / 8; i += kWave) {
      get8(i, f[0]);
#pragma unroll
      for (int q = 0; q < 8; ++q) peak_of(m, f[0][q]);
    }
  }
  int8_scale(__uint_as_float(wave_peak(m)), inv, sc);
  auto codes = [&](const float* v) {
    return make_uint2(i8x4(v[0], v[1], v[2], v[3], inv), i8x4(v[4], v[5], v[6], v[7], inv));
  };
  if (held) {
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (lane + p * kWave < n / 8) put2(lane + p * kWave, codes(f[p]));
  } else {
    for (int64_t i = lane; i < n / 8; i += kWave) {
      get8(i, f[0]);
      put2(i, codes(f[0]));
    }
  }
  return sc;
}

// Zeros behind rows of codes held in LDS, up to the end of the last step.
template <int THREADS>
__device__ __forceinline__ void held_pad(char* codes, int rows, int64_t n, int pitch) {
  const int pad = pitch - 64 - (int)n;  // a multiple of 8
  for (int i = threadIdx.x; i < rows * pad / 8; i += THREADS) {
    const int r = i / (pad / 8);
    *reinterpret_cast<uint2*>(codes + r * pitch + n + 8 * (i - r * (pad / 8))) = make_uint2(0u, 0u);
  }
}

// More than 64 KB of dynamic LDS has to be asked for, once for each kernel and device.
template <auto KERNEL>
bool lds_allowed(int bytes) {
  if (bytes <= 65536) return true;
  constexpr int kDevices = 64;
  static std::atomic<bool> asked[kDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return false;
  if (dev < kDevices && asked[dev].load(std::memory_order_relaxed)) return true;
  // (two threads may ask at once, both for all of it)
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize,
                          160 * 1024) != hipSuccess)
    return false;
  if (dev < kDevices) asked[dev].store(true, std::memory_order_relaxed);
  return true;
}

}  // namespace moe
