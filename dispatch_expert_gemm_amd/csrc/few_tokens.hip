// A whole MoE layer forward for a few tokens (T <= 64) in two kernels: every
// expert's weights are read from memory once, whatever the number of its rows,
// and nothing is rounded between x and out.
//
//   gate/up   for every active slot s = (t, k) of expert e:
//             h_s = silu(Wg_e x_t) * (Wu_e x_t)
//   down      out_t = bf16(sum_k w_tk v_tk + shared_t), v_tk = Wd_e h_s for a
//             routed slot, the special experts' values as in the combine
//
// There is no routing pass: each workgroup sorts the call's T K <= 1024 slots by
// expert in LDS for itself (route_lds).  A shared expert is one more expert that
// every token goes to with weight 1.
//
// Work split.  gate/up: a workgroup per (active expert, 16 columns of F), its
// waves splitting the contraction over H.  down: a workgroup per 16 columns of H
// that goes over all active experts, its waves splitting the (expert, F) steps
// evenly, so a token's weighted sum stays inside one workgroup: no atomics, and
// the same order of additions in every call.  Rows are packed per expert (the
// matrix cores take 16 at a time) and each wave adds its packed rows' weighted
// results to its own LDS copy of the output tile.
//
// bf16: h leaves as two bf16 planes, hi = bf16(h) and lo = bf16(h - hi), 16
// significant bits in all; both multiply the same weight registers.  int8: rows
// of x (times the expert's smooth scales) are quantised by a kernel before
// gate/up, rows of fp32 h by a kernel before down; sums are exact integers.
// Bound: HBM, the active experts' weights.
#include <initializer_list>

#include "combine_token.hpp"
#include "stream_mfma.hpp"

namespace moe {
namespace {

constexpr int kMaxTokens = 64, kMaxSlots = 1024, kMaxExperts = 1024;
constexpr int kUpWaves = 4, kDownWaves = 8;

struct FewArgs {
  const int32_t* idx;
  const float* w;
  const uint8_t* mask;
  const bf16_t* x;
  const void* wg;  // bf16 or int8 codes, (E, F, H)
  const void* wu;
  const void* wd;  // (E, H, F)
  const float* wgs;  // int8: one scale per output channel
  const float* wus;
  const float* wds;
  const void* swg;  // the shared expert's
  const void* swu;
  const void* swd;
  const float* swgs;
  const float* swus;
  const float* swds;
  const float* smooth;
  const bf16_t* shared_x;
  const bf16_t* a1;
  const bf16_t* a2;
  const bf16_t* cv;
  bf16_t* out;
  int32_t* err_flag;
  // workspace; rows of slots, then the shared expert's rows of tokens
  bf16_t* hhi;
  bf16_t* hlo;
  bf16_t* shhi;
  bf16_t* shlo;
  int8_t* xq;  // T rows of x, then T K rows of x * smooth
  float* xs;
  float* hf;
  float* shf;
  int8_t* hq;
  float* hs;
  int8_t* shq;
  float* shs;
  int64_t H, F, Fs;  // Fs 0: no shared expert
  int T, K, E, Z, C, Q, mask_ndim;
  int groups;  // most active experts: min(T K, E)
};

// The call's slots sorted by expert, in LDS.
struct Route {
  int32_t code[kMaxSlots];       // id of a routed slot, MOE_SLOT_NONE, MOE_SLOT_COPY or -(3 + j)
  int32_t first[kMaxExperts];    // slots of the expert, then the end of its run in `slot`
  uint16_t expert[kMaxSlots];    // active experts, in id order
  uint16_t begin[kMaxSlots + 1];  // the active expert's run in `slot`
  uint16_t slot[kMaxSlots];
  int32_t active;
  uint32_t err;
};

// Fills r (every thread of the workgroup; THREADS of them).  A masked, invalid
// or repeated slot (the later one) is inactive, as in the dispatch.  The order
// of an expert's slots in `slot` is not fixed; no result depends on it.
template <int THREADS>
__device__ void route_lds(const FewArgs& a, Route& r) {
  const int tid = threadIdx.x, S = a.T * a.K;
  for (int e = tid; e < a.E; e += THREADS) r.first[e] = 0;
  if (tid == 0) r.err = 0;
  for (int s = tid; s < S; s += THREADS) r.code[s] = a.idx[s];
  __syncthreads();
  int cls[(kMaxSlots + THREADS - 1) / THREADS];
  uint32_t err = 0;
#pragma unroll
  for (int i = 0; i < (kMaxSlots + THREADS - 1) / THREADS; ++i) {
    const int s = tid + i * THREADS;
    if (s >= S) break;
    const int t = s / a.K, k = s - t * a.K, id = r.code[s];
    bool act = true, dup = false;
    if (a.mask_ndim == 1) {
      act = a.mask[t] != 0;
      if (k == 0 && t > 0 && act && a.mask[t - 1] == 0) err |= MOE_FLAG_MASK_NOT_PREFIX;
    } else if (a.mask_ndim == 2) {
      act = a.mask[s] != 0;
    }
    for (int j = 1; j <= k; ++j) dup |= r.code[s - j] == id;
    int c = MOE_SLOT_NONE;
    if (id < 0 || id >= a.E + a.Z + a.C + a.Q) err |= MOE_FLAG_ID_RANGE;
    else if (dup) err |= MOE_FLAG_ID_DUPLICATE;
    else if (!act) ;
    else if (id < a.E) c = id;
    else if (id >= a.E + a.Z) c = id < a.E + a.Z + a.C ? MOE_SLOT_COPY : -(3 + (id - a.E - a.Z - a.C));
    cls[i] = c;
    if (c >= 0) atomicAdd(&r.first[c], 1);
  }
  if (err) atomicOr(&r.err, err);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < (kMaxSlots + THREADS - 1) / THREADS; ++i)
    if (tid + i * THREADS < S) r.code[tid + i * THREADS] = cls[i];
  if (tid < kWave) {
    // one wave: counts to run starts and the list of active experts
    int row = 0, n = 0;
    for (int base = 0; base < a.E; base += kWave) {
      const int e = base + tid, c = e < a.E ? r.first[e] : 0;
      int incl = c;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int v = __shfl_up(incl, o, kWave);
        if (tid >= o) incl += v;
      }
      const uint64_t m = __ballot(c > 0);
      if (c > 0) {
        const int at = n + __popcll(m & ((1ull << tid) - 1));
        r.expert[at] = (uint16_t)e;
        r.begin[at] = (uint16_t)(row + incl - c);
        r.first[e] = row + incl - c;
      }
      row += __shfl(incl, kWave - 1, kWave);
      n += __popcll(m);
    }
    if (tid == 0) {
      r.active = n;
      r.begin[n] = (uint16_t)row;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < (kMaxSlots + THREADS - 1) / THREADS; ++i) {
    const int s = tid + i * THREADS;
    if (s < S && cls[i] >= 0) r.slot[atomicAdd(&r.first[cls[i]], 1)] = (uint16_t)s;
  }
  __syncthreads();
}

// int8: one workgroup per row of codes: the tokens' rows, then (with smooth
// scales) the slots' rows x_t * smooth[e].  Slots that are not routed to an
// expert are left out.
__global__ __launch_bounds__(256) void k_few_quant_x(FewArgs a) {
  __shared__ float red[4];
  const int r = blockIdx.x;
  const float* sm = nullptr;
  int t = r;
  if (r >= a.T) {
    const int s = r - a.T, e = a.idx[s];
    if (e < 0 || e >= a.E) return;
    t = s / a.K;
    sm = a.smooth + (int64_t)e * a.H;
  } else if (a.smooth && a.Fs == 0) {
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H);
  uint2* dst = reinterpret_cast<uint2*>(a.xq + (int64_t)r * a.H);
  const float s = quant_row_int8<4>(
      a.H, red,
      [&](int64_t i, float* f) {
        unpack8(src[i], f);
        if (sm) {
#pragma unroll
          for (int q = 0; q < 8; ++q) f[q] = __fmul_rn(f[q], sm[8 * i + q]);
        }
      },
      [&](int64_t i, uint2 c) { dst[i] = c; });
  if (threadIdx.x == 0) a.xs[r] = s;
}

// int8: one workgroup per row of h: the slots' rows, then the shared expert's.
// Rows of slots that are not routed are unwritten, and never read.
__global__ __launch_bounds__(256) void k_few_quant_h(FewArgs a) {
  __shared__ float red[4];
  const int r = blockIdx.x, S = a.T * a.K;
  if (r < S && (a.idx[r] < 0 || a.idx[r] >= a.E)) return;
  const bool sh = r >= S;
  const int64_t n = sh ? a.Fs : a.F, row = sh ? r - S : r;
  const float4* src = reinterpret_cast<const float4*>((sh ? a.shf : a.hf) + row * n);
  uint2* dst = reinterpret_cast<uint2*>((sh ? a.shq : a.hq) + row * n);
  const float s = quant_row_int8<4>(
      n, red,
      [&](int64_t i, float* f) {
        const float4 p = src[2 * i], q = src[2 * i + 1];
        f[0] = p.x; f[1] = p.y; f[2] = p.z; f[3] = p.w;
        f[4] = q.x; f[5] = q.y; f[6] = q.z; f[7] = q.w;
      },
      [&](int64_t i, uint2 c) { dst[i] = c; });
  if (threadIdx.x == 0) (sh ? a.shs : a.hs)[row] = s;
}

// A group's rows r0 .. r0 + 16 RT - 1 through its 16 gate and 16 up columns from
// f0 on.  `slots`: the group's slots, NULL for the shared expert (row = token).
template <bool I8, int RT>
__device__ __forceinline__ void gate_up_rows(const FewArgs& a, const uint16_t* slots, int n, int r0, int e, int64_t f0,
                                             float4 (*red)[2][4][kWave]) {
  constexpr int ES = I8 ? 1 : 2;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  const int64_t F = sh ? a.Fs : a.F, bytes = a.H * ES;
  const int64_t wrow = (sh ? 0 : (int64_t)e * F) + f0;
  const int64_t woff = (wrow + lane % 16) * bytes + 16 * (lane / 16);
  const char* w[2] = {static_cast<const char*>(sh ? a.swg : a.wg) + woff, static_cast<const char*>(sh ? a.swu : a.wu) + woff};
  const char* x[1][RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int i = r0 + 16 * r + lane % 16;
    if (i >= n) i = n - 1;
    const int s = sh ? i : slots[i];
    const int64_t row = sh ? s : (I8 && a.smooth ? a.T + s : s / a.K);
    x[0][r] = (I8 ? reinterpret_cast<const char*>(a.xq) : reinterpret_cast<const char*>(a.x)) + row * bytes + 16 * (lane / 16);
  }
  typename MfmaAcc<I8>::type acc[2][RT];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[g][r] = typename MfmaAcc<I8>::type{0, 0, 0, 0};
  const int ns = stream_steps(bytes);
  stream_mfma<I8, 2, RT, 1, RT == 4 ? 2 : 4>(w, x, bytes, ns * wave / kUpWaves, ns * (wave + 1) / kUpWaves, acc);
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int r = 0; r < RT; ++r) red[wave][g][r][lane] = __builtin_bit_cast(float4, acc[g][r]);
  __syncthreads();
  const int i = r0 + 16 * wave + lane % 16;
  if (wave < RT && i < n) {
    typename MfmaAcc<I8>::type s[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      s[g] = __builtin_bit_cast(typename MfmaAcc<I8>::type, red[0][g][wave][lane]);
#pragma unroll
      for (int v = 1; v < kUpWaves; ++v)
        s[g] += __builtin_bit_cast(typename MfmaAcc<I8>::type, red[v][g][wave][lane]);
    }
    const int slot = sh ? i : slots[i];
    const int64_t c = 4 * (lane / 16), at = (int64_t)slot * F + f0 + c;
    float h[4];
    float xs = 1.f;
    if constexpr (I8) xs = a.xs[sh ? slot : (a.smooth ? a.T + slot : slot / a.K)];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float g = (float)s[0][q], u = (float)s[1][q];
      if constexpr (I8) {
        g *= __fmul_rn(xs, (sh ? a.swgs : a.wgs)[wrow + c + q]);
        u *= __fmul_rn(xs, (sh ? a.swus : a.wus)[wrow + c + q]);
      }
      h[q] = g / (1.0f + __expf(-g)) * u;
    }
    if constexpr (I8) {
      *reinterpret_cast<float4*>((sh ? a.shf : a.hf) + at) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
      float lo[4];
      uint32_t hi[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        hi[q] = f2bf(h[q]);
        // nothing below an infinite or NaN high part
        lo[q] = (hi[q] & 0x7f80u) == 0x7f80u ? 0.f : h[q] - bf2f(hi[q]);
      }
      *reinterpret_cast<uint2*>((sh ? a.shhi : a.hhi) + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>((sh ? a.shlo : a.hlo) + at) = make_uint2(pack_bf2(lo[0], lo[1]), pack_bf2(lo[2], lo[3]));
    }
  }
  __syncthreads();
}

template <bool I8>
__global__ __launch_bounds__(kUpWaves* kWave) void k_few_gate_up(FewArgs a) {
  __shared__ Route route;
  __shared__ float4 red[kUpWaves][2][4][kWave];
  route_lds<kUpWaves * kWave>(a, route);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err_flag = (int32_t)route.err;
  const int tiles = (int)(a.F / 16);
  const int g = blockIdx.x / tiles;
  const uint16_t* slots = nullptr;
  int n = a.T, e = 0;
  int64_t f0 = (int64_t)(blockIdx.x - a.groups * tiles) * 16;
  if (g < a.groups) {
    if (g >= route.active) return;
    e = route.expert[g];
    slots = route.slot + route.begin[g];
    n = route.begin[g + 1] - route.begin[g];
    f0 = (int64_t)(blockIdx.x % tiles) * 16;
  } else if (a.Fs == 0) {
    return;
  }
  for (int r0 = 0; r0 < n;) {
    const int left = (n - r0 + 15) / 16;
    if (left == 1) gate_up_rows<I8, 1>(a, slots, n, r0, e, f0, red);
    else if (left == 2) gate_up_rows<I8, 2>(a, slots, n, r0, e, f0, red);
    else gate_up_rows<I8, 4>(a, slots, n, r0, e, f0, red);
    r0 += left == 1 ? 16 : (left == 2 ? 32 : 64);
  }
}

// One expert's packed rows through this workgroup's 16 columns from c0 on, steps
// [s0, s1) of F, added to the wave's output tile `o` (T rows of 16 columns).
template <bool I8, int RT>
__device__ __forceinline__ void down_rows(const FewArgs& a, const uint16_t* slots, int n, int r0, int e, int64_t c0,
                                          int s0, int s1, float (*o)[16]) {
  constexpr int ES = I8 ? 1 : 2, PX = I8 ? 1 : 2;
  const int lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  const int64_t F = sh ? a.Fs : a.F, bytes = F * ES;
  const int64_t col = c0 + lane % 16 < a.H ? c0 + lane % 16 : a.H - 1;
  const int64_t wrow = sh ? 0 : (int64_t)e * a.H;
  const char* w[1] = {static_cast<const char*>(sh ? a.swd : a.wd) + (wrow + col) * bytes + 16 * (lane / 16)};
  const char* x[PX][RT];
  int slot[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int i = r0 + 16 * r + lane % 16;
    const bool in = i < n;
    if (!in) i = n - 1;
    const int s = sh ? i : slots[i];
    slot[r] = in ? s : -1;
    const int64_t off = s * bytes + 16 * (lane / 16);
    if constexpr (I8) {
      x[0][r] = reinterpret_cast<const char*>(sh ? a.shq : a.hq) + off;
    } else {
      x[0][r] = reinterpret_cast<const char*>(sh ? a.shhi : a.hhi) + off;
      x[1][r] = reinterpret_cast<const char*>(sh ? a.shlo : a.hlo) + off;
    }
  }
  typename MfmaAcc<I8>::type acc[1][RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[0][r] = typename MfmaAcc<I8>::type{0, 0, 0, 0};
  stream_mfma<I8, 1, RT, PX, RT == 1 ? 8 : (RT == 2 ? 4 : 2)>(w, x, bytes, s0, s1, acc);
  const int64_t c = c0 + 4 * (lane / 16);
  if (c >= a.H) return;  // H is a multiple of 8: four columns are in or out together
#pragma unroll
  for (int r = 0; r < RT; ++r)
    if (slot[r] >= 0) {
      const float wt = sh ? 1.0f : a.w[slot[r]];
      float4* p = reinterpret_cast<float4*>(&o[sh ? slot[r] : slot[r] / a.K][4 * (lane / 16)]);
      float4 v = *p;
      float y[4];
      float hs = 1.f;
      if constexpr (I8) hs = (sh ? a.shs : a.hs)[slot[r]];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        y[q] = (float)acc[0][r][q];
        if constexpr (I8) y[q] *= __fmul_rn(hs, (sh ? a.swds : a.wds)[wrow + c + q]);
      }
      v.x += wt * y[0]; v.y += wt * y[1]; v.z += wt * y[2]; v.w += wt * y[3];
      *p = v;
    }
  // the next expert's rows of the same tokens may sit in other lanes
  __builtin_amdgcn_wave_barrier();
}

// dynamic LDS: kDownWaves output tiles of T rows x 16 columns
template <bool I8>
__global__ __launch_bounds__(kDownWaves* kWave) void k_few_down(FewArgs a) {
  constexpr int ES = I8 ? 1 : 2;
  __shared__ Route route;
  extern __shared__ __attribute__((aligned(16))) float tiles[];
  const int wave = threadIdx.x / kWave;
  for (int i = threadIdx.x; i < kDownWaves * a.T * 16; i += kDownWaves * kWave) tiles[i] = 0.f;
  route_lds<kDownWaves * kWave>(a, route);
  const int64_t c0 = (int64_t)blockIdx.x * 16;
  float(*o)[16] = reinterpret_cast<float(*)[16]>(tiles) + wave * a.T;
  const int per = stream_steps(a.F * ES), routed = route.active * per;
  const int total = routed + stream_steps(a.Fs * ES);
  int u = (int)((int64_t)total * wave / kDownWaves);
  const int u1 = (int)((int64_t)total * (wave + 1) / kDownWaves);
  while (u < u1) {
    const bool sh = u >= routed;
    const int g = u / per, s0 = sh ? u - routed : u - g * per;
    const int len = (sh ? total - routed : per) - s0;
    const int s1 = s0 + (len < u1 - u ? len : u1 - u);
    const int n = sh ? a.T : route.begin[g + 1] - route.begin[g];
    const int e = sh ? 0 : route.expert[g];
    const uint16_t* slots = sh ? nullptr : route.slot + route.begin[g];
    for (int r0 = 0; r0 < n;) {
      const int left = (n - r0 + 15) / 16;
      if (left == 1) down_rows<I8, 1>(a, slots, n, r0, e, c0, s0, s1, o);
      else if (left == 2) down_rows<I8, 2>(a, slots, n, r0, e, c0, s0, s1, o);
      else down_rows<I8, 4>(a, slots, n, r0, e, c0, s0, s1, o);
      r0 += left == 1 ? 16 : (left == 2 ? 32 : 64);
    }
    u += s1 - s0;
  }
  __syncthreads();
  // join the waves' tiles, then the special experts in k order, the shared term last
  for (int i = threadIdx.x; i < a.T * 16; i += kDownWaves * kWave) {
    const int t = i / 16;
    const int64_t c = c0 + i % 16;
    if (c >= a.H) continue;
    float v = 0.f;
#pragma unroll
    for (int p = 0; p < kDownWaves; ++p) v += tiles[p * a.T * 16 + i];
    for (int k = 0; k < a.K; ++k) {
      const int code = route.code[t * a.K + k];
      if (code > MOE_SLOT_COPY) continue;
      float f = bf2f(a.x[t * a.H + c]);
      if (code != MOE_SLOT_COPY) {
        const int64_t j = (int64_t)(-code - 3) * a.H + c;
        f = bf2f(a.a1[j]) * f + bf2f(a.a2[j]) * bf2f(a.cv[j]);
      }
      v += a.w[t * a.K + k] * f;
    }
    if (a.shared_x) v += bf2f(a.shared_x[t * a.H + c]);
    a.out[t * a.H + c] = (bf16_t)f2bf(v);
  }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Places of the workspace's parts behind `base`; returns its size.
size_t few_layout(FewArgs& a, bool i8, char* base) {
  const size_t S = (size_t)a.T * a.K, T = a.T, H = a.H, F = a.F, Fs = a.Fs;
  size_t n = 0;
  auto take = [&](size_t bytes) {
    char* p = base + n;
    n += up256(bytes);
    return p;
  };
  if (i8) {
    a.xq = reinterpret_cast<int8_t*>(take((T + S) * H));
    a.xs = reinterpret_cast<float*>(take((T + S) * 4));
    a.hf = reinterpret_cast<float*>(take(S * F * 4));
    a.hq = reinterpret_cast<int8_t*>(take(S * F));
    a.hs = reinterpret_cast<float*>(take(S * 4));
    a.shf = reinterpret_cast<float*>(take(T * Fs * 4));
    a.shq = reinterpret_cast<int8_t*>(take(T * Fs));
    a.shs = reinterpret_cast<float*>(take(T * 4));
  } else {
    a.hhi = reinterpret_cast<bf16_t*>(take(S * F * 2));
    a.hlo = reinterpret_cast<bf16_t*>(take(S * F * 2));
    a.shhi = reinterpret_cast<bf16_t*>(take(T * Fs * 2));
    a.shlo = reinterpret_cast<bf16_t*>(take(T * Fs * 2));
  }
  return n < 256 ? 256 : n;
}

moe_status check_few(const moe_shape* s, int64_t shared_F, bool i8) {
  const moe_status st = check_ffn_shape(s);
  if (st != MOE_OK) return st;
  if (shared_F < 0 || shared_F % 32 != 0 || shared_F > (int64_t)1 << 20) return MOE_ERR_BAD_SHAPE;
  if (i8 && s->H % 16 != 0) return MOE_ERR_BAD_SHAPE;
  // |sum| <= 127 * 127 * (H or F) stays below 2^31
  if (i8 && (s->H > 131072 || s->F > 131072 || shared_F > 131072)) return MOE_ERR_UNSUPPORTED;
  if (s->comm_quant_mode != 0) return MOE_ERR_UNSUPPORTED;
  if (s->T > kMaxTokens) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// One expert weight tensor of either form.
struct FewWeight {
  const void* codes;
  const float* scales;
};

// The kernels read and write vectors of up to 16 bytes.
bool misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return true;
  return false;
}

moe_status few_impl(const moe_shape* s, bool i8, const void* x, const int32_t* topk_idx, const float* topk_weights,
                    const uint8_t* mask, const float* smooth, const FewWeight (&w)[3], int64_t Fs,
                    const FewWeight (&sw)[3], const void* shared_x, const void* a1, const void* a2, const void* cv,
                    void* out, int32_t* err_flag, void* workspace, size_t ws_bytes, hipStream_t strm) {
  const moe_status st = check_few(s, Fs, i8);
  if (st != MOE_OK) return st;
  if (!err_flag) return MOE_ERR_NULL_ARG;
  for (const FewWeight& v : w)
    if (!v.codes || (i8 && !v.scales)) return MOE_ERR_NULL_ARG;
  if (Fs > 0)
    for (const FewWeight& v : sw)
      if (!v.codes || (i8 && !v.scales)) return MOE_ERR_NULL_ARG;
  MOE_NEED(x, s->T);
  MOE_NEED(topk_idx, s->T);
  MOE_NEED(topk_weights, s->T);
  MOE_NEED(out, s->T);
  if (s->mask_ndim != 0) MOE_NEED(mask, s->T);
  if (Fs > 0 && shared_x) return MOE_ERR_BAD_RANGE;
  const moe_status sp = check_special(s, s->T ? x : (const void*)s, a1, a2, cv);
  if (sp != MOE_OK) return sp;
  if (misaligned({x, w[0].codes, w[1].codes, w[2].codes, sw[0].codes, sw[1].codes, sw[2].codes, workspace}))
    return MOE_ERR_BAD_SHAPE;
  FewArgs a = {};
  a.idx = topk_idx; a.w = topk_weights; a.mask = mask;
  a.x = static_cast<const bf16_t*>(x);
  a.wg = w[0].codes; a.wu = w[1].codes; a.wd = w[2].codes;
  a.wgs = w[0].scales; a.wus = w[1].scales; a.wds = w[2].scales;
  a.swg = sw[0].codes; a.swu = sw[1].codes; a.swd = sw[2].codes;
  a.swgs = sw[0].scales; a.swus = sw[1].scales; a.swds = sw[2].scales;
  a.smooth = smooth;
  a.shared_x = static_cast<const bf16_t*>(shared_x);
  a.a1 = static_cast<const bf16_t*>(a1); a.a2 = static_cast<const bf16_t*>(a2); a.cv = static_cast<const bf16_t*>(cv);
  a.out = static_cast<bf16_t*>(out);
  a.err_flag = err_flag;
  a.H = s->H; a.F = s->F; a.Fs = Fs;
  a.T = (int)s->T; a.K = s->K; a.E = s->num_experts;
  a.Z = s->zero_expert_num; a.C = s->copy_expert_num; a.Q = s->const_expert_num;
  a.mask_ndim = s->mask_ndim;
  const int S = a.T * a.K;
  a.groups = S < a.E ? S : a.E;
  const size_t need = few_layout(a, i8, static_cast<char*>(workspace));
  if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
  // gate/up tiles; one workgroup at least, for the error flag
  const int64_t nb = a.T == 0 ? 0 : a.groups * (a.F / 16) + Fs / 16;
  if (nb > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  const dim3 up((unsigned)(nb > 0 ? nb : 1)), down((unsigned)((a.H + 15) / 16));
  const size_t lds = (size_t)kDownWaves * a.T * 16 * 4;
  if (i8) {
    if (S > 0) hipLaunchKernelGGL(k_few_quant_x, dim3(a.T + (smooth ? S : 0)), dim3(256), 0, strm, a);
    hipLaunchKernelGGL(k_few_gate_up<true>, up, dim3(kUpWaves * kWave), 0, strm, a);
    if (S == 0) return launch_status();
    hipLaunchKernelGGL(k_few_quant_h, dim3(S + (Fs ? a.T : 0)), dim3(256), 0, strm, a);
    hipLaunchKernelGGL(k_few_down<true>, down, dim3(kDownWaves * kWave), lds, strm, a);
  } else {
    hipLaunchKernelGGL(k_few_gate_up<false>, up, dim3(kUpWaves * kWave), 0, strm, a);
    if (S == 0) return launch_status();
    hipLaunchKernelGGL(k_few_down<false>, down, dim3(kDownWaves * kWave), lds, strm, a);
  }
  return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_few_tokens_workspace_size(const moe_shape* s, int64_t shared_F, int32_t int8, size_t* bytes) {
  if (int8 != 0 && int8 != 1) return MOE_ERR_BAD_RANGE;
  const moe_status st = check_few(s, shared_F, int8 == 1);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_NULL_ARG;
  FewArgs a = {};
  a.T = (int)s->T; a.K = s->K; a.H = s->H; a.F = s->F; a.Fs = shared_F;
  *bytes = few_layout(a, int8 == 1, nullptr);
  return MOE_OK;
}

extern "C" moe_status moe_few_tokens(const moe_shape* s, const void* x, const int32_t* topk_idx,
                                     const float* topk_weights, const uint8_t* x_active_mask, const void* w_gate,
                                     const void* w_up, const void* w_down, int64_t shared_F, const void* shared_w_gate,
                                     const void* shared_w_up, const void* shared_w_down, const void* shared_expert_x,
                                     const void* const_alpha_1, const void* const_alpha_2, const void* const_v,
                                     void* out, int32_t* err_flag, void* workspace, size_t ws_bytes, void* stream) {
  return few_impl(s, false, x, topk_idx, topk_weights, x_active_mask, nullptr,
                  {{w_gate, nullptr}, {w_up, nullptr}, {w_down, nullptr}}, shared_F,
                  {{shared_w_gate, nullptr}, {shared_w_up, nullptr}, {shared_w_down, nullptr}}, shared_expert_x,
                  const_alpha_1, const_alpha_2, const_v, out, err_flag, workspace, ws_bytes, as_stream(stream));
}

extern "C" moe_status moe_few_tokens_int8(const moe_shape* s, const void* x, const int32_t* topk_idx,
                                          const float* topk_weights, const uint8_t* x_active_mask,
                                          const float* smooth_scales, const moe_int8_weight* w, int64_t shared_F,
                                          const moe_int8_weight* shared_w, const void* shared_expert_x,
                                          const void* const_alpha_1, const void* const_alpha_2, const void* const_v,
                                          void* out, int32_t* err_flag, void* workspace, size_t ws_bytes,
                                          void* stream) {
  if (!w || (shared_F > 0 && !shared_w)) return MOE_ERR_NULL_ARG;
  const moe_int8_weight none[3] = {};
  const moe_int8_weight* sw = shared_w ? shared_w : none;
  return few_impl(s, true, x, topk_idx, topk_weights, x_active_mask, smooth_scales,
                  {{w[0].codes, w[0].scales}, {w[1].codes, w[1].scales}, {w[2].codes, w[2].scales}}, shared_F,
                  {{sw[0].codes, sw[0].scales}, {sw[1].codes, sw[1].scales}, {sw[2].codes, sw[2].scales}},
                  shared_expert_x, const_alpha_1, const_alpha_2, const_v, out, err_flag, workspace, ws_bytes,
                  as_stream(stream));
}
