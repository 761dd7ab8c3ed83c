// Activation checkpoints in 8 bits (the rule in kept.hpp): SwiGLU whose [G | U] input
// is kept as int8 codes for the backward, and the combine whose expert rows are.
//
// All of it is bound by memory: each input is read once with 16-byte loads and
// each output written once.  On MI355X (a large copy moves 5.4 TB/s): SwiGLU of
// 65536 rows, F = 480, 45 us forward and 41 backward, 32768 rows, F = 2048, 97 and 97
// (5.6 TB/s); the combine of 8192 tokens, H = 1536, K = 8, 64 us (358 MB) and its
// weights' gradient 24 (132 MB).
#include <type_traits>

#include "combine_token.hpp"
#include "kept.hpp"

namespace moe {
namespace {

constexpr int kCols = kKeptCols;
constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

enum Pass : int { KEEP, GRAD };

struct SwigluArgs {
  const void* gate_up;   // KEEP: R x 2F
  const void* grad_h;    // GRAD: R x F
  const int32_t* nrows;  // rows in use, or NULL
  int8_t* codes;         // R x 2F
  uint16_t* scales;      // R x 2 x nb
  void* out;             // KEEP: h (R x F), GRAD: dG|dU (R x 2F)
  int64_t R, F, nb;
  // units of eight columns, `cols` of them a row of whole blocks
  uint32_t cols, step_rows, step_cols;  // kThreads units on: rows and columns
};

__device__ __forceinline__ int64_t rows_of(const SwigluArgs& a) {
  int64_t rows = a.R;
  if (a.nrows) {
    const int64_t n = *a.nrows;
    rows = n < 0 ? 0 : (n < rows ? n : rows);
  }
  return rows;
}

__device__ __forceinline__ uint4 pack8h(const float* f) {
  return make_uint4(pk_bf16(f[0], f[1]), pk_bf16(f[2], f[3]), pk_bf16(f[4], f[5]), pk_bf16(f[6], f[7]));
}

__device__ __forceinline__ void swiglu_grad(float g, float u, float d, float& dg, float& du) {
  const float sg = sigmoid(g), si = g * sg;
  dg = d * u * __fmaf_rn(si, 1.0f - sg, sg);
  du = d * si;
}

// Eight values of a row of F that begin at column c.  WHOLE: aligned, and all there.
// Otherwise the address may be any, and the row may end among the eight: they are
// then read as the row's last eight, and moved down (zeros behind) when they are
// used, so that every load goes out before the first wait.  A row of less than
// eight is read value by value.
template <bool WHOLE>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t c, int64_t F) {
  if (WHOLE) return *reinterpret_cast<const uint4*>(row + c);
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (F >= 8) {
    __builtin_memcpy(&v, row + (c < F - 8 ? c : F - 8), 16);
  } else if (c == 0) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < F) w[j / 2] |= (uint32_t)row[j] << (16 * (j & 1));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}
template <bool WHOLE>
__device__ __forceinline__ uint2 load8(const int8_t* row, int64_t c, int64_t F) {
  if (WHOLE) return *reinterpret_cast<const uint2*>(row + c);
  uint2 v = make_uint2(0u, 0u);
  if (F >= 8) {
    __builtin_memcpy(&v, row + (c < F - 8 ? c : F - 8), 8);
  } else if (c == 0) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < F) w[j / 4] |= (uint32_t)(uint8_t)row[j] << (8 * (j & 3));
    v = make_uint2(w[0], w[1]);
  }
  return v;
}
// n of the eight loaded: moved down by 8 - n (rows of less than eight came so).
__device__ __forceinline__ void settle8(uint4& v, int n, int64_t F) {
  if (n >= 8 || F < 8) return;
  const int k = 16 * (8 - n);  // 16 to 128 bits
  uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
  lo = k >= 64 ? (k == 128 ? 0ull : hi >> (k & 63)) : lo >> k | hi << (64 - k);
  hi = k >= 64 ? 0ull : hi >> k;
  v = make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
}
__device__ __forceinline__ void settle8(uint2& v, int n, int64_t F) {
  if (n >= 8 || F < 8) return;
  const int k = 8 * (8 - n);  // 8 to 64 bits
  uint64_t w = (uint64_t)v.y << 32 | v.x;
  w = k == 64 ? 0ull : w >> k;
  v = make_uint2((uint32_t)w, (uint32_t)(w >> 32));
}
// n of eight values to any address: 8, or 4, 2 and 1 of them.
// (The words are picked by value: picked by reference they would be an array in LDS,
// whose address takes the launch's packet in host memory, 14 us of a small call.)
template <bool WHOLE>
__device__ __forceinline__ void store8(uint16_t* p, uint4 v, int n) {
  if (WHOLE) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  if (n >= 8) {
    __builtin_memcpy(p, &v, 16);
    return;
  }
  const uint32_t x = v.x, y = v.y, z = v.z, w = v.w;
  const uint32_t two = n & 4 ? z : x, one = n & 4 ? (n & 2 ? w : z) : (n & 2 ? y : x);
  const uint2 four = make_uint2(x, y);
  if (n & 4) __builtin_memcpy(p, &four, 8);
  if (n & 2) __builtin_memcpy(p + (n & 4), &two, 4);
  if (n & 1) p[n & 6] = (uint16_t)one;
}
template <bool WHOLE>
__device__ __forceinline__ void store8(int8_t* p, uint2 v, int n) {
  if (WHOLE) {
    *reinterpret_cast<uint2*>(p) = v;
    return;
  }
  if (n >= 8) {
    __builtin_memcpy(p, &v, 8);
    return;
  }
  const uint32_t x = v.x, y = v.y, rest = n & 4 ? y : x;
  if (n & 4) __builtin_memcpy(p, &x, 4);
  const uint16_t two = (uint16_t)rest;
  if (n & 2) __builtin_memcpy(p + (n & 4), &two, 2);
  if (n & 1) p[n & 6] = (int8_t)(n & 2 ? rest >> 16 : rest);
}

// A lane takes eight columns of G and the same eight of U: a unit; U units a thread,
// kThreads apart, loads first.  WHOLE: F is a multiple of 32 and every matrix 16-byte
// aligned; otherwise a row is rounded up to whole blocks (units past F hold zeros) and
// accesses may begin anywhere (32768 rows of 1001 columns 44 us; a lane for each
// column 158).
template <int PASS, bool WHOLE, int U>
__global__ __launch_bounds__(kThreads) void k_swiglu_rows(SwigluArgs a) {
  constexpr int kUnits = U;
  const int64_t rows = rows_of(a), F = a.F;
  const int64_t u0 = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  int64_t row[kUnits];
  uint32_t col[kUnits];
  row[0] = u0 / a.cols;
  col[0] = (uint32_t)(u0 - row[0] * a.cols);
#pragma unroll
  for (int i = 1; i < kUnits; ++i) {
    row[i] = row[i - 1] + a.step_rows;
    col[i] = col[i - 1] + a.step_cols;
    if (col[i] >= a.cols) {
      col[i] -= a.cols;
      ++row[i];
    }
  }
  // columns of unit i that there are (8 where WHOLE), its place in a row of F
  auto count = [&](int i) {
    const int left = (int)F - 8 * (int)col[i];
    return WHOLE ? 8 : (left < 0 ? 0 : (left < 8 ? left : 8));
  };
  auto gate = [&](int i) { return row[i] * 2 * F + 8 * (int64_t)col[i]; };
  auto hcol = [&](int i) { return row[i] * F + 8 * (int64_t)col[i]; };
  if constexpr (PASS == KEEP) {
    const uint16_t* gu = static_cast<const uint16_t*>(a.gate_up);
    uint4 g[kUnits], u[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (row[i] < rows) {
        g[i] = load8<WHOLE>(gu + row[i] * 2 * F, 8 * (int64_t)col[i], F);
        u[i] = load8<WHOLE>(gu + row[i] * 2 * F + F, 8 * (int64_t)col[i], F);
      }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (row[i] >= rows) continue;  // the four lanes of a block leave together
      const int n = count(i);
      if constexpr (!WHOLE) {
        settle8(g[i], n, F);
        settle8(u[i], n, F);
      }
      float ig, iu;
      const uint32_t sg = kept_scale(block_amax(g[i]), ig), su = kept_scale(block_amax(u[i]), iu);
      store8<WHOLE>(a.codes + gate(i), codes8(g[i], ig), n);
      store8<WHOLE>(a.codes + gate(i) + F, codes8(u[i], iu), n);
      if ((col[i] & 3) == 0) {
        uint16_t* sc = a.scales + row[i] * 2 * a.nb + col[i] / 4;
        sc[0] = (uint16_t)sg;
        sc[a.nb] = (uint16_t)su;
      }
      float gf[8], uf[8];
      unpack8(g[i], gf);
      unpack8(u[i], uf);
#pragma unroll
      for (int j = 0; j < 8; ++j) gf[j] = gf[j] * sigmoid(gf[j]) * uf[j];
      store8<WHOLE>(static_cast<uint16_t*>(a.out) + hcol(i), pack8h(gf), n);
    }
  } else {
    uint2 qg[kUnits], qu[kUnits];
    uint32_t sg[kUnits], su[kUnits];
    uint4 dh[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (row[i] < rows) {
        const uint16_t* sc = a.scales + row[i] * 2 * a.nb + col[i] / 4;
        qg[i] = load8<WHOLE>(a.codes + row[i] * 2 * F, 8 * (int64_t)col[i], F);
        qu[i] = load8<WHOLE>(a.codes + row[i] * 2 * F + F, 8 * (int64_t)col[i], F);
        sg[i] = sc[0];
        su[i] = sc[a.nb];
        dh[i] = load8<WHOLE>(static_cast<const uint16_t*>(a.grad_h) + row[i] * F, 8 * (int64_t)col[i], F);
      }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (row[i] >= rows) continue;
      const int n = count(i);
      if constexpr (!WHOLE) {
        settle8(qg[i], n, F);
        settle8(qu[i], n, F);
        settle8(dh[i], n, F);
      }
      float g[8], u[8], d[8];
      kept8(qg[i], bf2f(sg[i]), g);
      kept8(qu[i], bf2f(su[i]), u);
      unpack8(dh[i], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) swiglu_grad(g[j], u[j], d[j], g[j], u[j]);
      uint16_t* out = static_cast<uint16_t*>(a.out) + gate(i);
      store8<WHOLE>(out, pack8h(g), n);
      store8<WHOLE>(out + F, pack8h(u), n);
    }
  }
}

// ----------------------------------------------------------------------------- combine

struct KeptArgs {
  uint2* codes;      // capacity x Hv, eight columns each
  uint16_t* scales;  // capacity x nb
  int64_t nb;
};

// Combine that keeps its rows: one wave for a token and a 64-vector column block
// (every split-th block), its routed rows' loads issued together; out is bit for
// bit k_combine's.  SPECIAL: copy or constant experts may be among the slots.
template <int KMAX, bool SPECIAL>
__global__ __launch_bounds__(kThreads) void k_combine_keep(CombineArgs a, KeptArgs q) {
#pragma clang fp contract(off)
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int64_t gw = (int64_t)blockIdx.x * (kThreads / kWave) + wave;
  const int64_t t = gw / a.split;
  const int part = (int)(gw - t * a.split);
  if (t >= a.T) return;
  SlotInfo<KMAX> si;
  load_slots(a.slot2row, a.w, t, a.K, lane, si);
  const int64_t Hv = a.Hv;
  for (int64_t b = part * kWave; b < Hv; b += (int64_t)a.split * kWave) {  // (the whole wave: blocks span lanes)
    const int64_t v = b + lane;
    const bool in = v < Hv;
    uint4 raw[KMAX], sh = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
      raw[k] = make_uint4(0u, 0u, 0u, 0u);
      if (si.code[k] >= 0 && in) raw[k] = ld_row(&a.y[(int64_t)si.code[k] * Hv + v]);
    }
    if (a.shared && in) sh = a.shared[t * Hv + v];
    float ox[8], acc[8];
    if (SPECIAL && si.any_ori && in) unpack8(a.ori[t * Hv + v], ox);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
      const int c = si.code[k];
      if (SPECIAL ? c == MOE_SLOT_NONE : c < 0) continue;
      float f[8];
      if (!SPECIAL || c >= 0) {
        float inv;
        const uint32_t s = kept_scale(block_amax(raw[k]), inv);
        const uint2 codes = codes8(raw[k], inv);
        if (in) {
          q.codes[(int64_t)c * Hv + v] = codes;
          if ((lane & 3) == 0) q.scales[(int64_t)c * q.nb + v / 4] = (uint16_t)s;
        }
        unpack8(raw[k], f);
      } else if (in) {
        special_value(c, ox, a.a1, a.a2, a.cv, Hv, v, f);
      }
      const float wk = si.w[k];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = acc[i] + wk * f[i];
    }
    if (in) {
      if (a.shared) {
        float sv[8];
        unpack8(sh, sv);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = acc[i] + sv[i];
      }
      a.out[t * Hv + v] = pack8(acc);
    }
  }
}

struct KeptBwdArgs {
  const uint4* dout;
  const uint2* codes;
  const uint16_t* scales;
  const float* w;
  const int32_t* slot2row;
  const uint4* ori;
  const uint4* a1;
  const uint4* a2;
  const uint4* cv;
  float* dw;
  float* roww;
  int64_t T, Hv, nb;
  int K;
};

// The routing weights' gradient from kept rows: W waves per token (1 or 4), each
// every W-th 64-vector column block, their sums joined in order.
template <int KMAX, bool SPECIAL, int W>
__global__ __launch_bounds__(kThreads) void k_combine_kept_bwd(KeptBwdArgs a) {
  constexpr int kTokens = kThreads / kWave / W;
  __shared__ float sums[kThreads / kWave][KMAX];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int part = W == 1 ? 0 : wave;
  const int64_t t = (int64_t)blockIdx.x * kTokens + (W == 1 ? wave : 0);
  if (t >= a.T) return;  // (with W = 4 the whole workgroup)
  SlotInfo<KMAX> si;
  load_slots(a.slot2row, a.w, t, a.K, lane, si);
  if (a.roww && part == 0)
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
      if (lane == k && si.code[k] >= 0) a.roww[si.code[k]] = si.w[k];
  const int64_t Hv = a.Hv;
  float dot[KMAX];
#pragma unroll
  for (int k = 0; k < KMAX; ++k) dot[k] = 0.f;
  for (int64_t v = part * kWave + lane; v < Hv; v += W * kWave) {
    uint2 raw[KMAX];
    uint32_t sc[KMAX];
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
      if (si.code[k] >= 0) {
        raw[k] = a.codes[(int64_t)si.code[k] * Hv + v];
        sc[k] = a.scales[(int64_t)si.code[k] * a.nb + v / 4];
      }
    float d[8];
    unpack8(a.dout[t * Hv + v], d);
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
      if (si.code[k] < 0) continue;
      // sum of code * d, then the scale: the eight codes share one
      float p = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        p = __fmaf_rn((float)(int8_t)((i < 4 ? raw[k].x : raw[k].y) >> (8 * (i & 3))), d[i], p);
      dot[k] = __fmaf_rn(p, bf2f(sc[k]), dot[k]);
    }
  }
  auto leave = [&](int k, float p) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) p += __shfl_xor(p, o, kWave);
    if (lane == 0) {
      if constexpr (W == 1) a.dw[t * a.K + k] = p;
      else sums[wave][k] = p;
    }
  };
#pragma unroll
  for (int k = 0; k < KMAX; ++k)
    if (k < a.K && (!SPECIAL || si.code[k] > MOE_SLOT_COPY)) leave(k, dot[k]);
  // copy and constant slots one after the other: among the routed ones they would
  // double the registers of the loop above (wide rows 68 -> 88 us)
  if (SPECIAL && si.any_ori)
    for (int k = 0; k < a.K; ++k) {
      const int c = __builtin_amdgcn_readfirstlane(a.slot2row[t * a.K + k]);
      if (c > MOE_SLOT_COPY) continue;
      float p = 0.f;
      for (int64_t v = part * kWave + lane; v < Hv; v += W * kWave) {
        float d[8], ox[8], f[8];
        unpack8(a.dout[t * Hv + v], d);
        unpack8(a.ori[t * Hv + v], ox);
        special_value(c, ox, a.a1, a.a2, a.cv, Hv, v, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) p = __fmaf_rn(f[i], d[i], p);
      }
      leave(k, p);
    }
  if constexpr (W > 1) {
    __syncthreads();
    const int k = threadIdx.x;
    if (k < a.K) {
      float p = sums[0][k];
#pragma unroll
      for (int w = 1; w < W; ++w) p += sums[w][k];
      a.dw[t * a.K + k] = p;
    }
  }
}

template <typename Fn>
inline void launch_k(int K, Fn f) {
  if (K <= 2) f(std::integral_constant<int, 2>{});
  else if (K <= 4) f(std::integral_constant<int, 4>{});
  else if (K <= 8) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

moe_status check_swiglu(int64_t R, int64_t F) {
  if (R < 0 || R > (int64_t)1 << 40 || F < 1 || F > (int64_t)1 << 20) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

constexpr int64_t kMaxWaves = kMaxThreads / kWave;

template <int PASS>
moe_status launch_swiglu(SwigluArgs a, void* stream) {
  a.nb = (a.F + kCols - 1) / kCols;
  const bool whole = a.F % kCols == 0 && aligned16(a.gate_up) && aligned16(a.grad_h) && aligned16(a.out) &&
                     reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  a.cols = (uint32_t)(a.nb * (kCols / 8));
  a.step_rows = kThreads / a.cols;
  a.step_cols = kThreads % a.cols;
  const int64_t units = a.R * (int64_t)a.cols;
  if (units / 2 > kMaxThreads) return MOE_ERR_UNSUPPORTED;
  auto go = [&](auto kernel, int per) {
    const int64_t each = per * kThreads;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((units + each - 1) / each)), dim3(kThreads), 0, as_stream(stream), a);
  };
  // two units a thread once that still gives every SIMD eight waves
  if (units < (int64_t)1 << 20) {
    if (whole) go(k_swiglu_rows<PASS, true, 1>, 1);
    else go(k_swiglu_rows<PASS, false, 1>, 1);
  } else {
    if (whole) go(k_swiglu_rows<PASS, true, 2>, 2);
    else go(k_swiglu_rows<PASS, false, 2>, 2);
  }
  return launch_status();
}

// Waves per token: one for each 64-vector column block, up to 16 and what a launch holds.
inline int keep_split(int64_t T, int64_t Hv) {
  int64_t split = (Hv + kWave - 1) / kWave;
  if (split > 16) split = 16;
  if (split > kMaxWaves / T) split = kMaxWaves / T;
  return (int)split;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_swiglu_checkpoint_fwd(int64_t R, int64_t F, const void* gate_up, const int32_t* nrows,
                                                void* h, int8_t* codes, void* scales, void* stream) {
  const moe_status st = check_swiglu(R, F);
  if (st != MOE_OK) return st;
  if (R == 0) return MOE_OK;
  if (!gate_up || !h || !codes || !scales) return MOE_ERR_NULL_ARG;
  SwigluArgs a{};
  a.gate_up = gate_up;
  a.nrows = nrows;
  a.codes = codes;
  a.scales = static_cast<uint16_t*>(scales);
  a.out = h;
  a.R = R;
  a.F = F;
  return launch_swiglu<KEEP>(a, stream);
}

extern "C" moe_status moe_swiglu_checkpoint_bwd(int64_t R, int64_t F, const int8_t* codes, const void* scales,
                                                const int32_t* nrows, const void* grad_h, void* grad_gate_up,
                                                void* stream) {
  const moe_status st = check_swiglu(R, F);
  if (st != MOE_OK) return st;
  if (R == 0) return MOE_OK;
  if (!codes || !scales || !grad_h || !grad_gate_up) return MOE_ERR_NULL_ARG;
  SwigluArgs a{};
  a.grad_h = grad_h;
  a.nrows = nrows;
  a.codes = const_cast<int8_t*>(codes);
  a.scales = static_cast<uint16_t*>(const_cast<void*>(scales));
  a.out = grad_gate_up;
  a.R = R;
  a.F = F;
  return launch_swiglu<GRAD>(a, stream);
}

extern "C" moe_status moe_combine_checkpoint(const moe_shape* s, const void* y, const int32_t* topk_idx,
                                             const float* topk_weights, const int32_t* assist,
                                             const int32_t* ep_send_counts, const uint8_t* x_active_mask,
                                             const void* shared_expert_x, const void* ori_x,
                                             const void* const_alpha_1, const void* const_alpha_2,
                                             const void* const_v, void* out, int8_t* y_codes, void* y_scales,
                                             void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->comm_quant_mode != 0) return MOE_ERR_UNSUPPORTED;
  if (s->T == 0) return MOE_OK;
  if (s->T > kMaxWaves) return MOE_ERR_UNSUPPORTED;
  MOE_NEED(y, s->capacity * s->H);
  MOE_NEED(y_codes, s->capacity * s->H);
  MOE_NEED(y_scales, s->capacity * s->H);
  if (!topk_idx || !topk_weights || !assist || !ep_send_counts || !out) return MOE_ERR_NULL_ARG;
  if (s->mask_ndim > 0 && !x_active_mask) return MOE_ERR_NULL_ARG;
  st = check_special(s, ori_x, const_alpha_1, const_alpha_2, const_v);
  if (st != MOE_OK) return st;
  const bool special = s->copy_expert_num + s->const_expert_num > 0;
  for (const void* p : {y, shared_expert_x, const_alpha_1, const_alpha_2, const_v, (const void*)out})
    if (!aligned16(p)) return MOE_ERR_BAD_SHAPE;
  if (special && !aligned16(ori_x)) return MOE_ERR_BAD_SHAPE;
  if (reinterpret_cast<uintptr_t>(y_codes) % 8) return MOE_ERR_BAD_SHAPE;
  const CombineArgs a{static_cast<const uint4*>(y),
                      topk_weights,
                      assist,
                      static_cast<const uint4*>(shared_expert_x),
                      static_cast<const uint4*>(ori_x),
                      static_cast<const uint4*>(const_alpha_1),
                      static_cast<const uint4*>(const_alpha_2),
                      static_cast<const uint4*>(const_v),
                      static_cast<uint4*>(out),
                      s->T,
                      s->K,
                      s->H / 8,
                      0,
                      keep_split(s->T, s->H / 8)};
  const KeptArgs q{reinterpret_cast<uint2*>(y_codes), static_cast<uint16_t*>(y_scales), (s->H + kCols - 1) / kCols};
  const int64_t waves = s->T * a.split;
  launch_k(s->K, [&](auto km) {
    constexpr int KM = decltype(km)::value;
    const dim3 grid((unsigned)((waves + 3) / 4));
    if (special)
      hipLaunchKernelGGL((k_combine_keep<KM, true>), grid, dim3(kThreads), 0, as_stream(stream), a, q);
    else
      hipLaunchKernelGGL((k_combine_keep<KM, false>), grid, dim3(kThreads), 0, as_stream(stream), a, q);
  });
  return launch_status();
}

extern "C" moe_status moe_combine_bwd_weights_checkpoint(
    const moe_shape* s, const void* grad_out, const int8_t* y_codes, const void* y_scales, const int32_t* topk_idx,
    const float* topk_weights, const int32_t* assist, const int32_t* ep_send_counts, const uint8_t* x_active_mask,
    const void* ori_x, const void* const_alpha_1, const void* const_alpha_2, const void* const_v,
    float* grad_topk_weights, float* row_weights, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->comm_quant_mode != 0) return MOE_ERR_UNSUPPORTED;
  if (s->T == 0) return MOE_OK;
  if (s->T > kMaxWaves) return MOE_ERR_UNSUPPORTED;
  MOE_NEED(y_codes, s->capacity * s->H);
  MOE_NEED(y_scales, s->capacity * s->H);
  if (!grad_out || !topk_idx || !topk_weights || !assist || !ep_send_counts || !grad_topk_weights)
    return MOE_ERR_NULL_ARG;
  if (s->mask_ndim > 0 && !x_active_mask) return MOE_ERR_NULL_ARG;
  st = check_special(s, ori_x, const_alpha_1, const_alpha_2, const_v);
  if (st != MOE_OK) return st;
  const bool special = s->copy_expert_num + s->const_expert_num > 0;
  for (const void* p : {grad_out, const_alpha_1, const_alpha_2, const_v})
    if (!aligned16(p)) return MOE_ERR_BAD_SHAPE;
  if (special && !aligned16(ori_x)) return MOE_ERR_BAD_SHAPE;
  if (reinterpret_cast<uintptr_t>(y_codes) % 8) return MOE_ERR_BAD_SHAPE;
  const KeptBwdArgs a{static_cast<const uint4*>(grad_out),
                      reinterpret_cast<const uint2*>(y_codes),
                      static_cast<const uint16_t*>(y_scales),
                      topk_weights,
                      assist,
                      static_cast<const uint4*>(ori_x),
                      static_cast<const uint4*>(const_alpha_1),
                      static_cast<const uint4*>(const_alpha_2),
                      static_cast<const uint4*>(const_v),
                      grad_topk_weights,
                      row_weights,
                      s->T,
                      s->H / 8,
                      (s->H + kCols - 1) / kCols,
                      s->K};
  launch_k(s->K, [&](auto km) {
    constexpr int KM = decltype(km)::value;
    auto go = [&](auto kernel, int64_t blocks) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, as_stream(stream), a);
    };
    // four waves for a row of four 64-vector blocks or more: 4096 tokens of 7168
    // columns 69 us against 75 with two (and 92 with one)
    if (a.Hv >= 256 && s->T <= kMaxWaves / 4) {
      if (special) go(k_combine_kept_bwd<KM, true, 4>, s->T);
      else go(k_combine_kept_bwd<KM, false, 4>, s->T);
    } else {
      if (special) go(k_combine_kept_bwd<KM, true, 1>, (s->T + 3) / 4);
      else go(k_combine_kept_bwd<KM, false, 1>, (s->T + 3) / 4);
    }
  });
  return launch_status();
}
