// A whole MoE layer forward for a few tokens (T <= 64): every expert's weights are
// read from memory once, whatever the number of its rows, and nothing is rounded
// between x and out.
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
// Work split.  gate/up: a workgroup per (active expert, columns of F), its waves
// splitting the contraction over H.  down, T <= 16: a workgroup per 32 columns of H
// that goes over all active experts, its waves splitting the (expert, F) steps
// evenly, so a token's weighted sum stays inside one workgroup: no third kernel, no
// atomics, the same order of additions in every call.  Rows are packed per expert
// (the matrix cores take 16 at a time); each wave adds its packed rows' weighted
// results to its own LDS copy of the output tile.  down, T > 16: a workgroup per
// (active expert, 64 columns), which reads each row of h half as often, and a
// small kernel for the weighted sums.
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

// Sizes of the work, by the row tiles (16 rows) that T tokens may need, RTM = 1, 2
// or 4.  Waves split the contraction; CT column tiles of a wave share its
// activation loads, which cost the vector L1 as much as the weights' (RT = 1 to 4
// tiles of rows, in bf16 two planes of h); U steps of loads are in flight in a
// wave.  (UP: gate/up, DN: down that sums over the experts, Y: down by expert.)
constexpr int kUpWaves = 4, kDownWaves = 8, kYWaves = 4;
template <int RTM>
constexpr int kUpCT = RTM == 1 ? 1 : 2;
template <int RTM>
constexpr int kDownCT = RTM == 1 ? 2 : 4;
template <int RTM>
constexpr int kUpOcc = RTM == 1 ? 4 : 2;  // waves per SIMD the registers have to leave room for
constexpr int kDownOcc = 3;
template <int RT>
constexpr int kUpU = RT == 4 ? 2 : 4;
template <int RT>
constexpr int kDownU = RT == 1 ? 4 : (RT == 2 ? 2 : 1);

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
  float* y;   // rows of slots, then the shared expert's: the expert outputs where down does not join them
};

// The call's slots sorted by expert, in LDS (sized by the call: route_bytes).
struct Route {
  int32_t* head;     // active experts, error bits
  int32_t* code;     // S: id of a routed slot, MOE_SLOT_NONE, MOE_SLOT_COPY or -(3 + j)
  int32_t* first;    // E: slots of the expert, then the end of its run in `slot`
  uint16_t* expert;  // active experts, in id order
  uint16_t* begin;   // the active expert's run in `slot`; one more than experts
  uint16_t* slot;    // S
};

__host__ __device__ inline int route_bytes(int S, int E, int groups) {
  const int n = 16 + 4 * (S + E) + 2 * (2 * groups + 1 + S);
  return (n + 15) / 16 * 16;
}

__device__ __forceinline__ Route route_at(char* lds, int S, int E, int groups) {
  Route r;
  r.head = reinterpret_cast<int32_t*>(lds);
  r.code = r.head + 4;
  r.first = r.code + S;
  r.expert = reinterpret_cast<uint16_t*>(r.first + E);
  r.begin = r.expert + groups;
  r.slot = r.begin + groups + 1;
  return r;
}

// Class of slot k of token t, `ids` its K ids: a routed expert's id, MOE_SLOT_NONE,
// MOE_SLOT_COPY or -(3 + j).  A masked, invalid or repeated slot (the later one) is
// inactive, as in the dispatch.
__device__ __forceinline__ int slot_code(const FewArgs& a, const int32_t* ids, int t, int k, uint32_t& err) {
  const int id = ids[k];
  bool act = true, dup = false;
  if (a.mask_ndim == 1) {
    act = a.mask[t] != 0;
    if (k == 0 && t > 0 && act && a.mask[t - 1] == 0) err |= MOE_FLAG_MASK_NOT_PREFIX;
  } else if (a.mask_ndim == 2) {
    act = a.mask[t * a.K + k] != 0;
  }
  for (int j = 0; j < k; ++j) dup |= ids[j] == id;
  if (id < 0 || id >= a.E + a.Z + a.C + a.Q) {
    err |= MOE_FLAG_ID_RANGE;
    return MOE_SLOT_NONE;
  }
  if (dup) {
    err |= MOE_FLAG_ID_DUPLICATE;
    return MOE_SLOT_NONE;
  }
  if (!act) return MOE_SLOT_NONE;
  if (id < a.E) return id;
  if (id < a.E + a.Z) return MOE_SLOT_NONE;
  return id < a.E + a.Z + a.C ? MOE_SLOT_COPY : -(3 + (id - a.E - a.Z - a.C));
}

// Fills r (every thread of the workgroup; THREADS of them, at most SLOTS slots).
// The order of an expert's slots in `slot` is not fixed; no result depends on it.
template <int THREADS, int SLOTS>
__device__ void route_lds(const FewArgs& a, const Route& r) {
  constexpr int PER = (SLOTS + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, S = a.T * a.K;
  int id[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) id[i] = tid + i * THREADS < S ? a.idx[tid + i * THREADS] : -1;
  for (int e = tid; e < a.E; e += THREADS) r.first[e] = 0;
  if (tid == 0) r.head[1] = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (tid + i * THREADS < S) r.code[tid + i * THREADS] = id[i];
  __syncthreads();
  uint32_t err = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = tid + i * THREADS;
    int c = MOE_SLOT_NONE;
    if (s < S) {
      const int t = s / a.K;
      c = slot_code(a, r.code + t * a.K, t, s - t * a.K, err);
      if (c >= 0) atomicAdd(&r.first[c], 1);
    }
    id[i] = c;
  }
  if (err) atomicOr(reinterpret_cast<uint32_t*>(&r.head[1]), err);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (tid + i * THREADS < S) r.code[tid + i * THREADS] = id[i];
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
      r.head[0] = n;
      r.begin[n] = (uint16_t)row;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (id[i] >= 0) r.slot[atomicAdd(&r.first[id[i]], 1)] = (uint16_t)(tid + i * THREADS);
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

// An expert's rows (at most 16 RT) through its 16 CT gate and 16 CT up columns from
// f0 on.  `slots`: the expert's slots, NULL for the shared expert (row = token).
// red: 2 RT KB for each wave.
template <bool I8, int RT, int CT>
__device__ __forceinline__ void gate_up_rows(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t f0,
                                             float4* red) {
  typedef typename MfmaAcc<I8>::type Acc;
  constexpr int ES = I8 ? 1 : 2, U = kUpU<RT>;
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  const int64_t F = sh ? a.Fs : a.F, bytes = a.H * ES;
  const int64_t wrow = (sh ? 0 : (int64_t)e * F) + f0;
  const char* w[2 * CT];
  uint32_t woff[2 * CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    // a column tile past F reads the first one
    const int64_t at = (wrow + (f0 + 16 * c < F ? 16 * c : 0)) * bytes;
    w[2 * c] = static_cast<const char*>(sh ? a.swg : a.wg) + at;
    w[2 * c + 1] = static_cast<const char*>(sh ? a.swu : a.wu) + at;
    woff[2 * c] = woff[2 * c + 1] = (uint32_t)(lane % 16) * (uint32_t)bytes + 16 * (lane / 16);
  }
  const char* x[1] = {I8 ? reinterpret_cast<const char*>(a.xq) : reinterpret_cast<const char*>(a.x)};
  uint32_t xoff[RT];  // at most 64 rows of 2^21 bytes, or 1088 of 2^17
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int i = 16 * r + lane % 16;
    if (i >= n) i = n - 1;
    const int s = sh ? i : slots[i];
    const int row = sh ? s : (I8 && a.smooth ? a.T + s : s / a.K);
    xoff[r] = (uint32_t)row * (uint32_t)bytes + 16 * (lane / 16);
  }
  Acc acc[2 * CT][RT];
#pragma unroll
  for (int g = 0; g < 2 * CT; ++g)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[g][r] = Acc{0, 0, 0, 0};
  const int ns = stream_steps(bytes);
  stream_mfma<I8, 2 * CT, RT, 1, U>(w, woff, x, xoff, bytes, ns * wave / kUpWaves, ns * (wave + 1) / kUpWaves, acc);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    if (ct > 0) __syncthreads();
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        red[((wave * 2 + g) * RT + r) * kWave + lane] = __builtin_bit_cast(float4, acc[2 * ct + g][r]);
    __syncthreads();
    const int r = wave;
    const int i = 16 * r + lane % 16;
    if (r >= RT || i >= n || f0 + 16 * ct >= F) continue;
    Acc s[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      s[g] = Acc{0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kUpWaves; ++v)
        s[g] += __builtin_bit_cast(Acc, red[((v * 2 + g) * RT + r) * kWave + lane]);
    }
    const int slot = sh ? i : slots[i];
    const int64_t c = 16 * ct + 4 * (lane / 16), at = (int64_t)slot * F + f0 + c;
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
}

// RTM: row tiles that T tokens may need (1, 2 or 4)
template <bool I8, int RTM, int CT>
__global__ __launch_bounds__(kUpWaves* kWave, kUpOcc<RTM>) void k_few_gate_up(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const Route route = route_at(lds, a.T * a.K, a.E, a.groups);
  float4* red = reinterpret_cast<float4*>(lds + route_bytes(a.T * a.K, a.E, a.groups));
  route_lds<kUpWaves * kWave, RTM * 256>(a, route);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err_flag = route.head[1];
  const int tiles = (int)((a.F + 16 * CT - 1) / (16 * CT));
  const int routed = uniform(route.head[0]) * tiles, items = routed + (int)((a.Fs + 16 * CT - 1) / (16 * CT));
  const int it = blockIdx.x;
  if (it < items) {
    const bool sh = it >= routed;
    const int g = sh ? 0 : it / tiles;
    const int b = sh ? 0 : uniform(route.begin[g]);
    const uint16_t* slots = sh ? nullptr : route.slot + b;
    const int n = sh ? a.T : uniform(route.begin[g + 1]) - b, e = sh ? 0 : uniform(route.expert[g]);
    const int64_t f0 = (int64_t)(sh ? it - routed : it - g * tiles) * (16 * CT);
    const int rt = (n + 15) / 16;
    if (RTM > 2 && rt > 2) gate_up_rows<I8, RTM, CT>(a, slots, n, e, f0, red);
    else if (RTM > 1 && rt > 1) gate_up_rows<I8, RTM < 2 ? 1 : 2, CT>(a, slots, n, e, f0, red);
    else gate_up_rows<I8, 1, CT>(a, slots, n, e, f0, red);
  }
}

// One expert's packed rows (at most 16 RT) through 16 CT columns of H from c0 on,
// steps [s0, s1) of F.  slot[r]: the lane's row (slot, or the shared expert's
// token), -1 past the last.
template <bool I8, int RT, int CT, int U>
__device__ __forceinline__ void down_stream(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t c0, int s0,
                                            int s1, int (&slot)[RT], typename MfmaAcc<I8>::type (&acc)[CT][RT]) {
  constexpr int ES = I8 ? 1 : 2, PX = I8 ? 1 : 2;
  const int lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  const int64_t F = sh ? a.Fs : a.F, bytes = F * ES;
  const int64_t wrow = sh ? 0 : (int64_t)e * a.H;
  const char* w[CT];
  uint32_t woff[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    // a column past H reads the last one
    const int64_t left = a.H - 1 - c0, col = 16 * c + lane % 16;
    w[c] = static_cast<const char*>(sh ? a.swd : a.wd) + (wrow + c0) * bytes;
    woff[c] = (uint32_t)(col < left ? col : left) * (uint32_t)bytes + 16 * (lane / 16);
  }
  const char* x[PX];
  x[0] = I8 ? reinterpret_cast<const char*>(sh ? a.shq : a.hq) : reinterpret_cast<const char*>(sh ? a.shhi : a.hhi);
  if constexpr (!I8) x[1] = reinterpret_cast<const char*>(sh ? a.shlo : a.hlo);
  uint32_t xoff[RT];  // at most 1024 rows of 2^21 bytes
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int i = 16 * r + lane % 16;
    const bool in = i < n;
    if (!in) i = n - 1;
    const int s = sh ? i : slots[i];
    slot[r] = in ? s : -1;
    xoff[r] = (uint32_t)s * (uint32_t)bytes + 16 * (lane / 16);
  }
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[c][r] = typename MfmaAcc<I8>::type{0, 0, 0, 0};
  stream_mfma<I8, CT, RT, PX, U>(w, woff, x, xoff, bytes, s0, s1, acc);
}

// down_stream of at most 16 rows, the weighted results added to the wave's output
// tile `o` (T rows of 16 CT columns).
template <bool I8, int CT>
__device__ __forceinline__ void down_rows(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t c0, int s0,
                                          int s1, float (*o)[16 * CT]) {
  const int lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  const int64_t wrow = sh ? 0 : (int64_t)e * a.H;
  typename MfmaAcc<I8>::type acc[CT][1];
  int slot[1];
  down_stream<I8, 1, CT, kDownU<1>>(a, slots, n, e, c0, s0, s1, slot, acc);
  if (slot[0] >= 0) {
    const float wt = sh ? 1.0f : a.w[slot[0]];
    float* row = o[sh ? slot[0] : slot[0] / a.K];
    float hs = 1.f;
    if constexpr (I8) hs = (sh ? a.shs : a.hs)[slot[0]];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int64_t c = c0 + 16 * ct + 4 * (lane / 16);
      if (c >= a.H) continue;  // H is a multiple of 8: four columns are in or out together
      float4* p = reinterpret_cast<float4*>(row + 16 * ct + 4 * (lane / 16));
      float4 v = *p;
      float y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        y[q] = (float)acc[ct][0][q];
        if constexpr (I8) y[q] *= __fmul_rn(hs, (sh ? a.swds : a.wds)[wrow + c + q]);
      }
      v.x += wt * y[0]; v.y += wt * y[1]; v.z += wt * y[2]; v.w += wt * y[3];
      *p = v;
    }
  }
  // the next expert's rows of the same tokens may sit in other lanes
  __builtin_amdgcn_wave_barrier();
}

// out[t, c] from its routed sum: the special experts in k order, the shared term last.
__device__ __forceinline__ void few_finish(const FewArgs& a, const int32_t* code, int t, int64_t c, float v) {
  for (int k = 0; k < a.K; ++k) {
    if (code[k] > MOE_SLOT_COPY) continue;
    float f = bf2f(a.x[t * a.H + c]);
    if (code[k] != MOE_SLOT_COPY) {
      const int64_t j = (int64_t)(-code[k] - 3) * a.H + c;
      f = bf2f(a.a1[j]) * f + bf2f(a.a2[j]) * bf2f(a.cv[j]);
    }
    v += a.w[t * a.K + k] * f;
  }
  if (a.shared_x) v += bf2f(a.shared_x[t * a.H + c]);
  a.out[t * a.H + c] = (bf16_t)f2bf(v);
}

// dynamic LDS: the routing, then kDownWaves output tiles of T rows x 16 CT columns
template <bool I8, int CT>
__global__ __launch_bounds__(kDownWaves* kWave, kDownOcc) void k_few_down(FewArgs a) {
  constexpr int ES = I8 ? 1 : 2, COLS = 16 * CT;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const Route route = route_at(lds, a.T * a.K, a.E, a.groups);
  float* tiles = reinterpret_cast<float*>(lds + route_bytes(a.T * a.K, a.E, a.groups));
  const int wave = uniform(threadIdx.x / kWave);
  for (int i = threadIdx.x; i < kDownWaves * a.T * COLS; i += kDownWaves * kWave) tiles[i] = 0.f;
  route_lds<kDownWaves * kWave, 256>(a, route);
  const int64_t c0 = (int64_t)blockIdx.x * COLS;
  float(*o)[COLS] = reinterpret_cast<float(*)[COLS]>(tiles) + wave * a.T;
  const int per = stream_steps(a.F * ES), routed = uniform(route.head[0]) * per;
  const int total = routed + stream_steps(a.Fs * ES);
  int u = (int)((int64_t)total * wave / kDownWaves);
  const int u1 = (int)((int64_t)total * (wave + 1) / kDownWaves);
  while (u < u1) {
    const bool sh = u >= routed;
    const int g = u / per, s0 = sh ? u - routed : u - g * per;
    const int len = (sh ? total - routed : per) - s0;
    const int s1 = s0 + (len < u1 - u ? len : u1 - u);
    const int b = sh ? 0 : uniform(route.begin[g]);
    const int n = sh ? a.T : uniform(route.begin[g + 1]) - b;
    const int e = sh ? 0 : uniform(route.expert[g]);
    const uint16_t* slots = sh ? nullptr : route.slot + b;
    u += s1 - s0;
    down_rows<I8, CT>(a, slots, n, e, c0, s0, s1, o);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * COLS; i += kDownWaves * kWave) {
    const int t = i / COLS;
    const int64_t c = c0 + i % COLS;
    if (c >= a.H) continue;
    float v = 0.f;
#pragma unroll
    for (int p = 0; p < kDownWaves; ++p) v += tiles[p * a.T * COLS + i];
    few_finish(a, route.code + t * a.K, t, c, v);
  }
}

// One expert's rows (at most 16 RT) through 16 CT columns of H from c0 on: rows of y.
// red: RT KB for each wave.
template <bool I8, int RT, int CT>
__device__ __forceinline__ void down_y_rows(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t c0,
                                            float4* red) {
  typedef typename MfmaAcc<I8>::type Acc;
  constexpr int U = kDownU<RT>;
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  Acc acc[CT][RT];
  int slot[RT];
  const int ns = stream_steps((sh ? a.Fs : a.F) * (I8 ? 1 : 2));
  down_stream<I8, RT, CT, U>(a, slots, n, e, c0, ns * wave / kYWaves, ns * (wave + 1) / kYWaves, slot, acc);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    if (ct > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r) red[(wave * RT + r) * kWave + lane] = __builtin_bit_cast(float4, acc[ct][r]);
    __syncthreads();
    const int i = 16 * wave + lane % 16;
    const int64_t c = c0 + 16 * ct + 4 * (lane / 16);
    if (wave >= RT || i >= n || c >= a.H) continue;
    Acc s = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kYWaves; ++v) s += __builtin_bit_cast(Acc, red[(v * RT + wave) * kWave + lane]);
    const int64_t row = sh ? i : slots[i];
    float y[4];
    float hs = 1.f;
    if constexpr (I8) hs = (sh ? a.shs : a.hs)[row];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      y[q] = (float)s[q];
      if constexpr (I8) y[q] *= __fmul_rn(hs, (sh ? a.swds : a.wds + (int64_t)e * a.H)[c + q]);
    }
    *reinterpret_cast<float4*>(a.y + (sh ? (int64_t)a.T * a.K + row : row) * a.H + c) = make_float4(y[0], y[1], y[2], y[3]);
  }
}

// larger batches: a workgroup per (active expert, 16 CT columns of H)
template <bool I8, int RTM, int CT>
__global__ __launch_bounds__(kYWaves* kWave, kDownOcc) void k_few_down_y(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const Route route = route_at(lds, a.T * a.K, a.E, a.groups);
  float4* red = reinterpret_cast<float4*>(lds + route_bytes(a.T * a.K, a.E, a.groups));
  route_lds<kYWaves * kWave, RTM * 256>(a, route);
  const int tiles = (int)((a.H + 16 * CT - 1) / (16 * CT));
  const int routed = uniform(route.head[0]) * tiles, items = routed + (a.Fs > 0 ? tiles : 0);
  const int it = blockIdx.x;
  if (it < items) {
    const bool sh = it >= routed;
    const int g = it / tiles;
    const int64_t c0 = (int64_t)(it - g * tiles) * (16 * CT);
    const int b = sh ? 0 : uniform(route.begin[g]);
    const uint16_t* slots = sh ? nullptr : route.slot + b;
    const int n = sh ? a.T : uniform(route.begin[g + 1]) - b, e = sh ? 0 : uniform(route.expert[g]);
    const int rt = (n + 15) / 16;
    if (RTM > 2 && rt > 2) down_y_rows<I8, RTM, CT>(a, slots, n, e, c0, red);
    else if (RTM > 1 && rt > 1) down_y_rows<I8, RTM < 2 ? 1 : 2, CT>(a, slots, n, e, c0, red);
    else down_y_rows<I8, 1, CT>(a, slots, n, e, c0, red);
  }
}

// four outputs of one token per thread: the weighted sum of y over its slots in k
// order, the shared expert's row and the shared term
__global__ __launch_bounds__(256) void k_few_join(FewArgs a) {
  __shared__ int32_t code[16];
  const int t = blockIdx.y;
  if (threadIdx.x < a.K) {
    uint32_t err = 0;
    code[threadIdx.x] = slot_code(a, a.idx + t * a.K, t, threadIdx.x, err);
  }
  __syncthreads();
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (c >= a.H) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k <= a.K; ++k) {
    const bool sh = k == a.K;
    if (sh ? a.Fs == 0 : code[k] < 0) continue;
    const float wt = sh ? 1.f : a.w[t * a.K + k];
    const float4 y = *reinterpret_cast<const float4*>(a.y + (sh ? (int64_t)a.T * a.K + t : (int64_t)t * a.K + k) * a.H + c);
    v[0] += wt * y.x; v[1] += wt * y.y; v[2] += wt * y.z; v[3] += wt * y.w;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) few_finish(a, code, t, c + q, v[q]);
}

// Whether the down kernel sums over the experts itself (two kernels in all).
bool few_joins(int T) { return T <= 16; }

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
  if (!few_joins(a.T)) a.y = reinterpret_cast<float*>(take((S + T) * H * 4));
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

template <bool I8, int RTM>
moe_status few_launch(FewArgs& a, hipStream_t strm) {
  constexpr int UC = kUpCT<RTM>, DC = kDownCT<RTM>;
  const int S = a.T * a.K, rb = route_bytes(S, a.E, a.groups);
  auto tiles = [](int64_t n, int ct) { return (n + 16 * ct - 1) / (16 * ct); };
  const int64_t up = a.groups * tiles(a.F, UC) + tiles(a.Fs, UC);
  if (up > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((k_few_gate_up<I8, RTM, UC>), dim3((unsigned)up), dim3(kUpWaves * kWave),
                     rb + kUpWaves * 2 * RTM * kWave * 16, strm, a);
  if (I8) hipLaunchKernelGGL(k_few_quant_h, dim3(S + (a.Fs ? a.T : 0)), dim3(256), 0, strm, a);
  if constexpr (RTM == 1) {
    hipLaunchKernelGGL((k_few_down<I8, DC>), dim3((unsigned)tiles(a.H, DC)), dim3(kDownWaves * kWave),
                       rb + kDownWaves * a.T * 16 * DC * 4, strm, a);
  } else {
    hipLaunchKernelGGL((k_few_down_y<I8, RTM, DC>), dim3((unsigned)(a.groups + (a.Fs > 0)) * tiles(a.H, DC)),
                       dim3(kYWaves * kWave), rb + kYWaves * RTM * kWave * 16, strm, a);
    hipLaunchKernelGGL(k_few_join, dim3((unsigned)((a.H + 1023) / 1024), (unsigned)a.T), dim3(256), 0, strm, a);
  }
  return launch_status();
}

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
  if (S == 0) {
    // the error flag alone
    a.Fs = 0;
    hipLaunchKernelGGL((k_few_gate_up<false, 1, kUpCT<1>>), dim3(1), dim3(kUpWaves * kWave), route_bytes(0, a.E, 0), strm, a);
    return launch_status();
  }
  if (i8) {
    hipLaunchKernelGGL(k_few_quant_x, dim3(a.T + (smooth ? S : 0)), dim3(256), 0, strm, a);
    return a.T <= 16 ? few_launch<true, 1>(a, strm) : (a.T <= 32 ? few_launch<true, 2>(a, strm) : few_launch<true, 4>(a, strm));
  }
  return a.T <= 16 ? few_launch<false, 1>(a, strm) : (a.T <= 32 ? few_launch<false, 2>(a, strm) : few_launch<false, 4>(a, strm));
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
