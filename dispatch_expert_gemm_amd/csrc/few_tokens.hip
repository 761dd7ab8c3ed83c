// A whole MoE layer forward for a few tokens (T <= 64): every expert's weights are
// read from memory once, whatever the number of its rows, and nothing is rounded
// below fp32 between x and out (int8: but to the codes).
//
//   gate/up   for every active slot s = (t, k) of expert e:
//             h_s = silu(Wg_e x_t) * (Wu_e x_t)
//   down      out_t = bf16(sum_k w_tk v_tk + shared_t), v_tk = Wd_e h_s for a
//             routed slot, the special experts' values as in the combine
//
// A shared expert is one more expert that every token goes to with weight 1.
//
// Kernels.  T <= 16: k_few_gate_up, k_few_down, or for narrow layers k_few_down_y and
// k_few_join in the latter's place (few_joins).  T > 16: k_few_prep, k_few_gate_up,
// k_few_down_y, k_few_join.  int8 has its rows quantised by k_few_prep (x, times the
// expert's smooth scales) and k_few_quant_h (h); one or two tokens (HELD) form the
// codes inside the two kernels that use them.
//
// Route.  The T K <= 1024 slots sorted by expert: with T <= 16 every workgroup of
// gate/up sorts them in LDS for itself (no launch), and the first leaves the table for
// the kernels behind; with more k_few_prep does it once.
//
// Split.  gate/up: a workgroup per (active expert, columns of F); a long contraction over
// H is split over its four waves, a short one is one wave's own.  down, T <= 16: a
// workgroup per 16 or 32 columns of H that goes over all active experts, its eight waves
// splitting the (expert, F) steps evenly, so a token's weighted sum stays inside one
// workgroup: no third kernel, no atomics, the same order of additions in every call (where
// a wave's steps begin follows from the number of active experts, so the other tokens'
// ids may change the order, their values do not).
// Rows are packed per expert (the matrix cores take 16 at a time); each wave adds its
// packed rows' weighted results to its own LDS copy of the output tile.  down, T > 16: a
// workgroup per (active expert, columns of H), which reads each row of h less often, and
// a small kernel for the weighted sums, again in a fixed order.
//
// Every operand of a product goes straight into LDS, in whole cache lines, by loads that
// have no register result; each wave has a ring of a few steps for itself and waits by
// count, so the main loops have no barrier (stream_mfma.hpp).
//
// bf16: h leaves in fp32, and its three bf16 parts, every bit of it, multiply the same
// weight registers.  int8: sums are exact integers,
// those of k_few_down over a wave's part of F, and the parts join in fp32.
//
// Bound: HBM, the active experts' weights (reads reach 6.0 TB/s here).  Layers on
// MI355X with cold weights: one token, 8 of 32 experts and a shared one, H = 7168,
// F = 2048: 147 us, 5.4 TB/s (int8 85 us, 4.7); 13 tokens 461 us, 5.8 TB/s (9 in int8 224 us,
// 5.6); 64 tokens on 8 experts of 14336 x 4096 498 us, 5.7 TB/s (each expert's rows 64
// of them, top 8: 714 us); 64 tokens in int8 309 us, 4.7.  One token of 64 experts of 1536 x
// 480: 16.6 us, of which the bytes are 6.
#include <cmath>
#include <initializer_list>

#include "combine_token.hpp"
#include "stream_mfma.hpp"

namespace moe {
namespace {

constexpr int kMaxTokens = 64, kMaxSlots = 1024;

// Sizes of the work.  Up: gate/up, Down: down that sums over the experts, Y: down by
// expert.  A wave's ring of LDS holds D steps of its operands; CT column tiles of a
// wave share its activation rows.  Up's ring, up to 16 rows for an expert: 8 KB takes one
// token with a shared expert from 146 to 154 us, 24 KB 9 tokens in int8 from 228 to 263
// (fewer workgroups on a CU); more rows: 12 KB takes 64 tokens in int8 from 308 to 315, 24 KB
// to 334.
constexpr int kUpWaves = 4, kDownWaves = 8, kYWaves = 4;
template <int RTM>
constexpr int kUpRing = RTM == 1 ? 12288 : 16384;
// 128-byte steps of H below which a wave has its columns to itself, and steps of F likewise
// (Y).  Split at every length: 48 tokens on 64 experts of 1536 x 480 in int8 47 -> 64 us;
// split at none: 64 tokens on 8 experts of 4096 x 14336 501 -> 562 us, one token 17 -> 19.
constexpr int kUpOwn = 16, kYOwn = 40;
// (8 KB: 2 tokens of 64 experts of 1536 x 512 in bf16 25.5 -> 27.0 us; 16 KB: 13 tokens of 32
// experts of 7168 x 2048 458 -> 463 us, others equal)
constexpr int kDownRing = 12288;
// Y, by the waves KS that split the contraction: a long one wants few reads of h
// (64 tokens of 8 experts of F = 14336 in bf16: the layer 505 us, with two column tiles 534;
// with top 8 714 against 813), a short one more workgroups on a CU, whose beginnings and
// ends overlap (48 tokens of 64 experts of F = 480 in int8: 47.4 us, with four column
// tiles 53.8)
template <int KS>
constexpr int kYCT = KS == 1 ? 2 : 4;
template <bool I8, int RTM, int KS>
constexpr int kYRing = KS > 1 ? 24576 : (I8 || RTM < 4 ? 12288 : 20480);
template <int NW, int RT, int PX, int RING>
constexpr int kDepth = RING / kSlot<NW, RT, PX> < 1 ? 1 : (RING / kSlot<NW, RT, PX> > 4 ? 4 : RING / kSlot<NW, RT, PX>);
// int8, one or two tokens: the rows' codes are formed by the kernels that use them, which
// saves two launches (one token of 64 experts of 1536 x 512 20.6 -> 15.8 us, two of 5120 x
// 1536 48 -> 43.6; two of 7168 x 2048 with a shared expert 134.7 -> 136.7).  Four tokens: 27.7
// against 26.0 us with the launches.  A ring of three steps in gate/up leaves a workgroup
// less on a CU: 87 -> 92.6 us.
constexpr int kHeldTokens = 2, kHeldUpDepth = 2, kHeldDownDepth = 3, kHeldBytes = 49152;

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
  char* table;  // workspace: the route
  // workspace; rows of slots, then the shared expert's rows of tokens
  float* h[2];   // bf16: fp32 rows in two planes
  float* sh[2];
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

// The call's slots sorted by expert.
struct Route {
  int32_t* head;     // active experts, error bits
  int32_t* code;     // S: id of a routed slot, MOE_SLOT_NONE, MOE_SLOT_COPY or -(3 + j)
  uint16_t* expert;  // active experts, in id order
  uint16_t* begin;   // the active expert's run in `slot`; one more than experts
  uint16_t* slot;    // S
  int32_t* first;    // E, while it is built: slots of the expert, then the end of its run
};

// Bytes of a route without `first` (a multiple of 16), and with it.
__host__ __device__ inline int route_bytes(int S, int groups) {
  return (16 + 4 * S + 2 * (2 * groups + 1 + S) + 15) / 16 * 16;
}
__host__ __device__ inline int route_work_bytes(int S, int E, int groups) {
  return (route_bytes(S, groups) + 4 * E + 15) / 16 * 16;
}

__device__ __forceinline__ Route route_at(char* p, int S, int groups) {
  Route r;
  r.head = reinterpret_cast<int32_t*>(p);
  r.code = r.head + 4;
  r.expert = reinterpret_cast<uint16_t*>(r.code + S);
  r.begin = r.expert + groups;
  r.slot = r.begin + groups + 1;
  r.first = reinterpret_cast<int32_t*>(p + route_bytes(S, groups));
  return r;
}

// A whole route, copied by every thread of the workgroup (THREADS of them).
template <int THREADS>
__device__ __forceinline__ void route_copy(char* to, const char* from, int S, int groups) {
  for (int i = threadIdx.x; i < route_bytes(S, groups) / 16; i += THREADS)
    reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(from)[i];
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

// Fills r in LDS (every thread of the workgroup; THREADS of them, at most SLOTS slots).
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

// Values 8 i .. 8 i + 7 of a row of x, times its smooth scales (NULL: 1).
__device__ __forceinline__ void x_times_smooth(const uint4& x, const float* smooth, int64_t i, float* f) {
  unpack8(x, f);
  if (!smooth) return;
  const float4 p = reinterpret_cast<const float4*>(smooth)[2 * i], q = reinterpret_cast<const float4*>(smooth)[2 * i + 1];
  f[0] = __fmul_rn(f[0], p.x); f[1] = __fmul_rn(f[1], p.y); f[2] = __fmul_rn(f[2], p.z); f[3] = __fmul_rn(f[3], p.w);
  f[4] = __fmul_rn(f[4], q.x); f[5] = __fmul_rn(f[5], q.y); f[6] = __fmul_rn(f[6], q.z); f[7] = __fmul_rn(f[7], q.w);
}

// The first workgroup routes the call for the kernels behind it (ROUTE); int8: one
// more for each row of codes: the tokens' rows, then (with smooth scales) the slots'
// rows x_t * smooth[e].  Slots that are not routed to an expert are left out.
template <bool ROUTE, bool I8>
__global__ __launch_bounds__(256) void k_few_prep(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  if (ROUTE && blockIdx.x == 0) {
    const Route r = route_at(lds, a.T * a.K, a.groups);
    route_lds<256, kMaxSlots>(a, r);
    if (threadIdx.x == 0) *a.err_flag = r.head[1];
    route_copy<256>(a.table, lds, a.T * a.K, a.groups);
  }
  if constexpr (I8) {
    const int r = (int)blockIdx.x - (ROUTE ? 1 : 0);
    const float* sm = nullptr;
    int t = r;
    if (r < 0) return;
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
        a.H, reinterpret_cast<uint32_t*>(lds),
        [&](int64_t i, float* f) {
          x_times_smooth(src[i], sm, i, f);
        },
        [&](int64_t i, uint2 c) { dst[i] = c; });
    if (threadIdx.x == 0) a.xs[r] = s;
  }
}

// Values 8 i .. 8 i + 7 of a fp32 row.
__device__ __forceinline__ void load8(const float4* src, int64_t i, float* f) {
  const float4 p = src[2 * i], q = src[2 * i + 1];
  f[0] = p.x; f[1] = p.y; f[2] = p.z; f[3] = p.w;
  f[4] = q.x; f[5] = q.y; f[6] = q.z; f[7] = q.w;
}

// int8: one workgroup per row of h: the slots' rows, then the shared expert's.
// Rows of slots that are not routed are unwritten, and never read.
template <int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void k_few_quant_h(FewArgs a) {
  __shared__ uint32_t red[WAVES];
  const int r = blockIdx.x, S = a.T * a.K;
  if (r < S && (a.idx[r] < 0 || a.idx[r] >= a.E)) return;
  const bool sh = r >= S;
  const int64_t n = sh ? a.Fs : a.F, row = sh ? r - S : r;
  const float4* src = reinterpret_cast<const float4*>((sh ? a.shf : a.hf) + row * n);
  uint2* dst = reinterpret_cast<uint2*>((sh ? a.shq : a.hq) + row * n);
  const float s = quant_row_int8<WAVES>(
      n, red,
      [&](int64_t i, float* f) {
        load8(src, i, f);
      },
      [&](int64_t i, uint2 c) { dst[i] = c; });
  if (threadIdx.x == 0) (sh ? a.shs : a.hs)[row] = s;
}

// Offsets of an expert's packed rows in a matrix of `bytes`-byte rows: tile r's row
// stream_row(j) is row_of(16 r + stream_row(j)); rows past n read zeros.
template <int RT, int XI, class F>
__device__ __forceinline__ void row_offsets(int n, int64_t bytes, uint32_t (&xoff)[RT][XI], F row_of) {
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < XI; ++j) {
      const int i = 16 * r + stream_row(j);
      xoff[r][j] = i < n ? (uint32_t)row_of(i) * (uint32_t)bytes : kPastBuffer;
    }
}

// G and U of four columns of one row (int8: of scale xs) -> h from column c on.
template <bool I8>
__device__ __forceinline__ void swiglu_store(const FewArgs& a, bool sh, int slot, float xs, int64_t wrow, int64_t c,
                                             const typename MfmaAcc<I8>::type& sg, const typename MfmaAcc<I8>::type& su) {
  const int64_t F = sh ? a.Fs : a.F;
  float h[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float g = (float)sg[q], u = (float)su[q];
    if constexpr (I8) {
      g *= __fmul_rn(xs, (sh ? a.swgs : a.wgs)[wrow + q]);
      u *= __fmul_rn(xs, (sh ? a.swus : a.wus)[wrow + q]);
    }
    h[q] = g / (1.0f + __expf(-g)) * u;
  }
  float* at = I8 ? (sh ? a.shf : a.hf) + (int64_t)slot * F + c : plane_at(sh ? a.sh : a.h, F, slot, c);
  *reinterpret_cast<float4*>(at) = make_float4(h[0], h[1], h[2], h[3]);
}

// An expert's rows (at most 16 RT, XI = 1: 8) through its gate and up columns from f0
// on, 16 of each for every KS waves, which split the contraction.  `slots`: the
// expert's slots, NULL for the shared expert (row = token).  lds: the waves' rings.
template <bool I8, int RT, int XI, int KS, int RING>
__device__ __forceinline__ void gate_up_rows(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t f0,
                                             char* lds) {
  typedef typename MfmaAcc<I8>::type Acc;
  constexpr int ES = I8 ? 1 : 2;
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  const int64_t F = sh ? a.Fs : a.F, bytes = a.H * ES;
  f0 += 16 * (wave / KS);
  const bool in = f0 < F;  // (KS < waves: the last workgroup's waves may have no columns)
  const int64_t wrow = (sh ? 0 : (int64_t)e * F) + (in ? f0 : 0);
  const i32x4_t w[2] = {buffer_of(static_cast<const char*>(sh ? a.swg : a.wg) + wrow * bytes, 16 * bytes),
                        buffer_of(static_cast<const char*>(sh ? a.swu : a.wu) + wrow * bytes, 16 * bytes)};
  auto x_row = [&](int s) { return sh ? s : (I8 && a.smooth ? a.T + s : s / a.K); };
  const i32x4_t x[1] = {I8 ? buffer_of(a.xq, (a.T + (a.smooth ? a.T * a.K : 0)) * bytes) : buffer_of(a.x, a.T * bytes)};
  uint32_t xoff[RT][XI];
  row_offsets<RT, XI>(n, bytes, xoff, [&](int i) { return x_row(sh ? i : slots[i]); });
  Acc acc[2][RT];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[g][r] = Acc{0, 0, 0, 0};
  const int ns = in ? stream_steps(bytes) : 0, part = wave % KS;
  static_assert(kSlot<2, RT, 1> <= RING, "a ring holds a step");
  stream_mfma<I8, 2, RT, 1, XI, kDepth<2, RT, 1, RING>>(w, x, xoff, bytes, ns * part / KS, ns * (part + 1) / KS,
                                                          lds + wave * RING, acc);
  const int64_t c = 4 * (lane / 16);
  auto finish = [&](int r, const Acc& g, const Acc& u) {
    const int i = 16 * r + lane % 16;
    if (!in || i >= n) return;
    const int slot = sh ? i : slots[i];
    swiglu_store<I8>(a, sh, slot, I8 ? a.xs[x_row(slot)] : 1.f, wrow + c, f0 + c, g, u);
  };
  if constexpr (KS == 1) {
#pragma unroll
    for (int r = 0; r < RT; ++r) finish(r, acc[0][r], acc[1][r]);
  } else {
    static_assert(KS == kUpWaves && RT <= KS && 2 * RT * 1024 <= RING, "parts");
    // the waves' parts meet in their rings' place
    float4* red = reinterpret_cast<float4*>(lds);
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        red[wave * (RING / 16) + (g * RT + r) * kWave + lane] = __builtin_bit_cast(float4, acc[g][r]);
    __syncthreads();
    if (wave < RT) {
      Acc s[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        s[g] = Acc{0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < KS; ++v)
          s[g] += __builtin_bit_cast(Acc, red[v * (RING / 16) + (g * RT + wave) * kWave + lane]);
      }
      finish(wave, s[0], s[1]);
    }
  }
}

// gate_up_rows for one or two tokens in int8: the rows are quantised here, behind the
// first weight loads (every workgroup of an expert does it again: a launch of its own
// costs about 5 us).  lds: the waves' rings, the codes, scales and maxima.
__device__ __forceinline__ void gate_up_held(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t f0,
                                             char* lds) {
  constexpr int W = kUpWaves, RING = kHeldUpDepth * kSlot<2, 0, 0>;
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, pitch = held_pitch(a.H);
  const bool sh = slots == nullptr;
  const int64_t F = sh ? a.Fs : a.F, wrow = (sh ? 0 : (int64_t)e * F) + f0;
  char* codes = lds + W * RING;
  float* scales = reinterpret_cast<float*>(codes + a.T * pitch);
  uint32_t* red = reinterpret_cast<uint32_t*>(scales + kHeldTokens);
  const i32x4_t w[2] = {buffer_of(static_cast<const char*>(sh ? a.swg : a.wg) + wrow * a.H, 16 * a.H),
                        buffer_of(static_cast<const char*>(sh ? a.swu : a.wu) + wrow * a.H, 16 * a.H)};
  i32x4_t acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  const int ns = stream_steps(a.H), mine = lane % 16 < n ? lane % 16 : 0;
  const float* sm = sh || !a.smooth ? nullptr : a.smooth + (int64_t)e * a.H;
  stream_held<2, kHeldUpDepth>(w, codes + mine * pitch + 16 * (lane / 16), a.H, ns * wave / W, ns * (wave + 1) / W,
                               lds + wave * RING, acc, [&] {
    quant_rows_int8<W, kHeldTokens, 4>(
        n, a.H, red,
        [&](int r, int64_t i, float* f) {
          const int t = sh ? r : slots[r] / a.K;
          x_times_smooth(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H)[i], sm, i, f);
        },
        [&](int r, int64_t i, uint2 c) { *reinterpret_cast<uint2*>(codes + r * pitch + 8 * i) = c; },
        [&](int r, float s) { scales[r] = s; });
    held_pad<W * kWave>(codes, n, a.H, pitch);
    __syncthreads();
  });
  i32x4_t* red2 = reinterpret_cast<i32x4_t*>(lds);
#pragma unroll
  for (int g = 0; g < 2; ++g) red2[wave * (RING / 16) + g * kWave + lane] = acc[g];
  __syncthreads();
  if (wave > 0 || lane % 16 >= n) return;
  i32x4_t s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int v = 0; v < W; ++v) s[g] += red2[v * (RING / 16) + g * kWave + lane];
  const int slot = sh ? mine : slots[mine];
  const int64_t c = 4 * (lane / 16);
  swiglu_store<true>(a, sh, slot, scales[mine], wrow + c, f0 + c, s[0], s[1]);
}

// RTM: row tiles that T tokens may need (1, 2 or 4).  RTM = 1 routes for itself, and
// the first workgroup for the kernels behind it.
template <bool I8, int RTM, int KS, bool HELD>
__global__ __launch_bounds__(kUpWaves* kWave, 2) void k_few_gate_up(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int COLS = 16 * kUpWaves / KS;
  const int S = a.T * a.K;
  const Route route = route_at(RTM == 1 ? lds : a.table, S, a.groups);
  char* rings = lds + (RTM == 1 ? route_work_bytes(S, a.E, a.groups) : 0);
  if constexpr (RTM == 1) {
    route_lds<kUpWaves * kWave, 256>(a, route);
    if (blockIdx.x == 0) {
      if (threadIdx.x == 0) *a.err_flag = route.head[1];
      route_copy<kUpWaves * kWave>(a.table, lds, S, a.groups);
    }
  }
  const int tiles = (int)((a.F + COLS - 1) / COLS);
  const int routed = uniform(route.head[0]) * tiles, items = routed + (int)((a.Fs + COLS - 1) / COLS);
  const int it = blockIdx.x;
  if (it >= items) return;
  const bool sh = it >= routed;
  const int g = sh ? 0 : it / tiles;
  const int b = sh ? 0 : uniform(route.begin[g]);
  const uint16_t* slots = sh ? nullptr : route.slot + b;
  const int n = sh ? a.T : uniform(route.begin[g + 1]) - b, e = sh ? 0 : uniform(route.expert[g]);
  const int64_t f0 = (int64_t)(sh ? it - routed : it - g * tiles) * COLS;
  if constexpr (HELD) {
    gate_up_held(a, slots, n, e, f0, rings);
  } else {
    constexpr int RING = kUpRing<RTM>;
    const int rt = (n + 15) / 16;
    if (RTM > 2 && rt > 2) gate_up_rows<I8, RTM, 2, KS, RING>(a, slots, n, e, f0, rings);
    else if (RTM > 1 && rt > 1) gate_up_rows<I8, RTM < 2 ? 1 : 2, 2, KS, RING>(a, slots, n, e, f0, rings);
    else if (n > 8) gate_up_rows<I8, 1, 2, KS, RING>(a, slots, n, e, f0, rings);
    else gate_up_rows<I8, 1, 1, KS, RING>(a, slots, n, e, f0, rings);
  }
}

// Column tile c from c0 on of an expert's W_down: columns past H lie past the buffer, a
// tile past H reads the first one.
__device__ __forceinline__ i32x4_t down_weights(const FewArgs& a, bool sh, int e, int64_t c0, int c, int64_t bytes) {
  const int64_t col = c0 + (c0 + 16 * c < a.H ? 16 * c : 0), left = a.H - col;
  return buffer_of(static_cast<const char*>(sh ? a.swd : a.wd) + ((sh ? 0 : (int64_t)e * a.H) + col) * bytes,
                   (left < 16 ? left : 16) * bytes);
}

// One expert's packed rows (at most 16 RT, XI = 1: 8) through 16 CT columns of H from
// c0 on, steps [s0, s1) of F.
template <bool I8, int RT, int XI, int CT, int RING>
__device__ __forceinline__ void down_stream(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t c0, int s0,
                                            int s1, char* ring, typename MfmaAcc<I8>::type (&acc)[CT][RT]) {
  constexpr int ES = I8 ? 1 : 2, PX = I8 ? 1 : 2;
  const bool sh = slots == nullptr;
  const int64_t F = sh ? a.Fs : a.F, bytes = F * ES, pitch = I8 ? F : plane_pitch(F);
  const int64_t rows = sh ? a.T : (int64_t)a.T * a.K;
  i32x4_t w[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    w[c] = down_weights(a, sh, e, c0, c, bytes);
  }
  i32x4_t x[PX];
  if constexpr (I8) {
    x[0] = buffer_of(sh ? a.shq : a.hq, rows * pitch);
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) x[p] = buffer_of(sh ? a.sh[p] : a.h[p], rows * pitch);
  }
  uint32_t xoff[RT][XI];
  row_offsets<RT, XI>(n, pitch, xoff, [&](int i) { return sh ? i : (int)slots[i]; });
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[c][r] = typename MfmaAcc<I8>::type{0, 0, 0, 0};
  static_assert(kSlot<CT, RT, PX> <= RING, "a ring holds a step");
  stream_mfma<I8, CT, RT, PX, XI, kDepth<CT, RT, PX, RING>>(w, x, xoff, bytes, s0, s1, ring, acc);
}

// int8, one or two tokens: the codes of every row of h in LDS (slots, then the shared
// expert's), and their scales.
struct HeldRows {
  char* codes;
  float* scales;
};
__host__ __device__ inline int held_h_bytes(int S, int T, int64_t F, int64_t Fs) {
  return S * held_pitch(F) + (Fs ? T * held_pitch(Fs) : 0);
}
__device__ __forceinline__ int held_h_at(int S, int64_t F, int64_t Fs, bool sh, int row) {
  return sh ? S * held_pitch(F) + row * held_pitch(Fs) : row * held_pitch(F);
}

// down_stream of at most 16 rows, the weighted results added to the wave's output
// tile `o` (T rows of 16 CT columns).  XI = 0: the rows are in LDS (held).
template <bool I8, int XI, int CT, int RING>
__device__ __forceinline__ void down_rows(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t c0, int s0,
                                          int s1, char* ring, float (*o)[16 * CT], const HeldRows& held) {
  const int lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  const int64_t wrow = sh ? 0 : (int64_t)e * a.H;
  const int row = lane % 16 < n ? (sh ? lane % 16 : slots[lane % 16]) : -1;
  float wt = 1.f, hs = 1.f;
  if (row >= 0) {
    if (!sh) wt = a.w[row];
    if constexpr (XI == 0) hs = held.scales[sh ? a.T * a.K + row : row];
    else if constexpr (I8) hs = (sh ? a.shs : a.hs)[row];
  }
  typename MfmaAcc<I8>::type acc[CT][1];
  if constexpr (XI == 0) {
    const int64_t bytes = sh ? a.Fs : a.F;
    const int any = row >= 0 ? row : (sh ? 0 : slots[0]);
    i32x4_t w[CT], sum[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      w[c] = down_weights(a, sh, e, c0, c, bytes);
      sum[c] = i32x4_t{0, 0, 0, 0};
    }
    stream_held<CT, RING / kSlot<CT, 0, 0>>(w, held.codes + held_h_at(a.T * a.K, a.F, a.Fs, sh, any) + 16 * (lane / 16), bytes, s0,
                                    s1, ring, sum, [] {});
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c][0] = sum[c];
  } else {
    down_stream<I8, 1, XI, CT, RING>(a, slots, n, e, c0, s0, s1, ring, acc);
  }
  if (row >= 0) {
    float* out = o[sh ? row : row / a.K];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int64_t c = c0 + 16 * ct + 4 * (lane / 16);
      if (c >= a.H) continue;  // H is a multiple of 8: four columns are in or out together
      float4* p = reinterpret_cast<float4*>(out + 16 * ct + 4 * (lane / 16));
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

// dynamic LDS: the routing, the waves' rings and output tiles of T rows x 16 CT columns
template <bool I8, int CT, bool HELD>
__global__ __launch_bounds__(kDownWaves* kWave, 2) void k_few_down(FewArgs a) {
  constexpr int ES = I8 ? 1 : 2, COLS = 16 * CT;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const Route route = route_at(lds, a.T * a.K, a.groups);
  constexpr int RING = HELD ? kHeldDownDepth * kSlot<CT, 0, 0> : kDownRing;
  const int S = a.T * a.K;
  char* rings = lds + route_bytes(S, a.groups);
  float* tiles = reinterpret_cast<float*>(rings + kDownWaves * RING);
  const int wave = uniform(threadIdx.x / kWave);
  for (int i = threadIdx.x; i < kDownWaves * a.T * COLS; i += kDownWaves * kWave) tiles[i] = 0.f;
  route_copy<kDownWaves * kWave>(lds, a.table, S, a.groups);
  HeldRows held = {};
  if constexpr (HELD) {
    // every row of h to int8, a wave a row
    held.scales = tiles + kDownWaves * a.T * COLS;
    held.codes = reinterpret_cast<char*>(held.scales + (S + a.T + 3) / 4 * 4);
    const Route table = route_at(a.table, S, a.groups);
    for (int r = wave; r < S + (a.Fs ? a.T : 0); r += kDownWaves) {
      const bool sh = r >= S;
      if (!sh && uniform(table.code[r]) < 0) continue;
      const int row = sh ? r - S : r;
      const int64_t n = sh ? a.Fs : a.F;
      const float4* src = reinterpret_cast<const float4*>((sh ? a.shf : a.hf) + row * n);
      char* dst = held.codes + held_h_at(S, a.F, a.Fs, sh, row);
      const float sc = quant_row_int8_wave(
          n, [&](int64_t i, float* f) { load8(src, i, f); },
          [&](int64_t i, uint2 c) { *reinterpret_cast<uint2*>(dst + 8 * i) = c; });
      const int lane = threadIdx.x % kWave;
      if (lane == 0) held.scales[r] = sc;
      // zeros up to the end of the last step
      for (int64_t i = n + 8 * lane; i < held_pitch(n) - 64; i += 8 * kWave) *reinterpret_cast<uint2*>(dst + i) = make_uint2(0u, 0u);
    }
  }
  __syncthreads();
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
    if constexpr (HELD) down_rows<I8, 0, CT, RING>(a, slots, n, e, c0, s0, s1, rings + wave * RING, o, held);
    else if (n > 8) down_rows<I8, 2, CT, RING>(a, slots, n, e, c0, s0, s1, rings + wave * RING, o, held);
    else down_rows<I8, 1, CT, RING>(a, slots, n, e, c0, s0, s1, rings + wave * RING, o, held);
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

// One expert's rows (at most 16 RT) through columns of H from c0 on, 16 kYCT for every
// KS waves, which split the contraction: rows of y.  lds: the waves' rings.
template <bool I8, int RTM, int RT, int XI, int KS>
__device__ __forceinline__ void down_y_rows(const FewArgs& a, const uint16_t* slots, int n, int e, int64_t c0,
                                            char* lds) {
  typedef typename MfmaAcc<I8>::type Acc;
  constexpr int CT = kYCT<KS>, RING = kYRing<I8, RTM, KS>;
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const bool sh = slots == nullptr;
  c0 += 16 * CT * (wave / KS);
  const bool in = c0 < a.H;
  Acc acc[CT][RT];
  const int ns = in ? stream_steps((sh ? a.Fs : a.F) * (I8 ? 1 : 2)) : 0, part = wave % KS;
  down_stream<I8, RT, XI, CT, RING>(a, slots, n, e, in ? c0 : 0, ns * part / KS, ns * (part + 1) / KS,
                                      lds + wave * RING, acc);
  auto finish = [&](int ct, int r, const Acc& s) {
    const int i = 16 * r + lane % 16;
    const int64_t c = c0 + 16 * ct + 4 * (lane / 16);
    if (i >= n || c >= a.H) return;
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
  };
  if constexpr (KS == 1) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int r = 0; r < RT; ++r) finish(ct, r, acc[ct][r]);
  } else {
    static_assert(KS == kYWaves && CT * RT * 1024 <= RING, "parts");
    float4* red = reinterpret_cast<float4*>(lds);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        red[wave * (RING / 16) + (ct * RT + r) * kWave + lane] = __builtin_bit_cast(float4, acc[ct][r]);
    __syncthreads();
    for (int q = wave; q < CT * RT; q += KS) {
      Acc s = {0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < KS; ++v) s += __builtin_bit_cast(Acc, red[v * (RING / 16) + q * kWave + lane]);
      finish(q / RT, q % RT, s);
    }
  }
}

// larger batches: a workgroup per (active expert, columns of H)
template <bool I8, int RTM, int KS>
__global__ __launch_bounds__(kYWaves* kWave, 2) void k_few_down_y(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int COLS = 16 * kYCT<KS> * kYWaves / KS;
  const Route route = route_at(a.table, a.T * a.K, a.groups);
  const int tiles = (int)((a.H + COLS - 1) / COLS);
  const int routed = uniform(route.head[0]) * tiles, items = routed + (a.Fs > 0 ? tiles : 0);
  const int it = blockIdx.x;
  if (it >= items) return;
  const bool sh = it >= routed;
  const int g = it / tiles;
  const int64_t c0 = (int64_t)(it - g * tiles) * COLS;
  const int b = sh ? 0 : uniform(route.begin[g]);
  const uint16_t* slots = sh ? nullptr : route.slot + b;
  const int n = sh ? a.T : uniform(route.begin[g + 1]) - b, e = sh ? 0 : uniform(route.expert[g]);
  const int rt = (n + 15) / 16;
  if (RTM > 2 && rt > 2) down_y_rows<I8, RTM, RTM, 2, KS>(a, slots, n, e, c0, lds);
  else if (RTM > 1 && rt > 1) down_y_rows<I8, RTM, RTM < 2 ? 1 : 2, 2, KS>(a, slots, n, e, c0, lds);
  else if (n > 8) down_y_rows<I8, RTM, 1, 2, KS>(a, slots, n, e, c0, lds);
  else down_y_rows<I8, RTM, 1, 1, KS>(a, slots, n, e, c0, lds);
}

// four outputs of one token per thread: the weighted sum of y over its slots in k
// order, the shared expert's row, the special experts and the shared term
template <int KMAX>
__global__ __launch_bounds__(256) void k_few_join(FewArgs a) {
  const int t = blockIdx.y;
  const int32_t* code = route_at(a.table, a.T * a.K, a.groups).code + t * a.K;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (c >= a.H) return;
  // every slot's row is read at once, also those that nothing was written to, and used
  // or not afterwards
  float4 y[KMAX + 1];
  int cd[KMAX];
  float wt[KMAX];
#pragma unroll
  for (int k = 0; k < KMAX; ++k)
    if (k < a.K) {
      y[k] = *reinterpret_cast<const float4*>(a.y + ((int64_t)t * a.K + k) * a.H + c);
      cd[k] = code[k];
      wt[k] = a.w[t * a.K + k];
    }
  if (a.Fs > 0) y[KMAX] = *reinterpret_cast<const float4*>(a.y + ((int64_t)a.T * a.K + t) * a.H + c);
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k <= KMAX; ++k) {
    if (k < KMAX ? k >= a.K || cd[k < KMAX ? k : 0] < 0 : a.Fs == 0) continue;
    const float w = k < KMAX ? wt[k < KMAX ? k : 0] : 1.f;
    v[0] += w * y[k].x; v[1] += w * y[k].y; v[2] += w * y[k].z; v[3] += w * y[k].w;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) few_finish(a, code, t, c + q, v[q]);
}

// int8: whether the rows are quantised inside the two kernels.
bool few_held(const FewArgs& a, bool i8) {
  return i8 && a.T <= kHeldTokens && a.H <= 4 * 8 * kUpWaves * kWave &&
         held_h_bytes(a.T * a.K, a.T, a.F, a.Fs) <= kHeldBytes;
}

// Whether the down kernel sums over the experts itself: its H / 16 workgroups, each over
// all active experts, against workgroups by expert and a launch for the sums.  A narrow
// layer has too few of the former.  Both are estimated (us) for slots spread evenly over
// the experts, with rates fitted to what they measure: itself, 38 bytes per ns of 16 columns
// and 0.15 us for each expert's beginning; by expert, the longest workgroup or 5 TB/s in
// all, and 5 us for the launch.  Itself / by expert, measured, the whole layer (us):
//   64 experts of 1536 x 480, top 8   bf16  1 token 17.2 / 20.5, 4 39.6 / 36.2, 16 76.7 / 60.9
//                                     int8  4 tokens 28.9 / 29.5, 6 38.6 / 36.0, 16 53.6 / 43.8
//   38 of 672 x 3744, top 4           bf16  3 tokens 73 / 49.5, 6 118 / 66
//                                     int8  3 tokens 47.0 / 45.3, 6 74.7 / 57.9
//   3584 x 2048, 16 tokens of 16, top 8     bf16 139.9 / 142.6, int8 82.8 / 84.7
//                8 tokens of 8, top 2       bf16 60.3 / 71.7, int8 44.2 / 45.7
//   128 of 2048 x 768, top 8          bf16  16 tokens 168 / 148, 4 67.1 / 60.8
//                                     int8  16 tokens 111 / 101, 4 49.9 / 46.7
// The estimate takes the lesser but for the 4 tokens of 128 experts (10 and 7% more) and 4 int8
// tokens of 64 (2%).
bool few_joins(const FewArgs& a, bool i8) {
  if (a.T > 16) return false;
  if (a.H > 16 * 256 || few_held(a, i8)) return true;
  const double es = i8 ? 1 : 2, active = a.E * (1 - std::exp(-(double)a.T * a.K / a.E));
  const double bytes = (active * (double)a.F + a.Fs) * es;  // of one column
  const double itself = bytes * 16 / 38e3 + 0.15 * active;
  // one workgroup by expert: 128 columns with a step or two of loads under way, or 64 with more
  const bool own = stream_steps((int64_t)(a.F * es)) < kYOwn;
  const double one = a.F * es * (own ? 128 / (i8 ? 45e3 : 25e3) : 64 / 60e3);
  return itself <= std::fmax(one, bytes * a.H / 5e6) + 5;
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
  a.table = take(route_bytes((int)S, a.groups));
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
    for (float*& p : a.h) p = reinterpret_cast<float*>(take(S * plane_pitch(F)));
    for (float*& p : a.sh) p = reinterpret_cast<float*>(take(T * plane_pitch(Fs)));
  }
  if (!few_joins(a, i8)) a.y = reinterpret_cast<float*>(take((S + T) * H * 4));
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
  // the rows of h (of a plane, F * 2 bytes and at most 64 more, or of codes) are addressed
  // with 31-bit offsets: 1024 of them of F <= 2^20 - 32 end at 2^31 (those of x below 2^27)
  if (s->T * s->K * s->F * 2 >= 0x7ffffff0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// One expert weight tensor of either form.
struct FewWeight {
  const void* codes;
  const float* scales;
};

// Waves that split gate/up's contraction: all for a long one, a short one is a wave's own.
int up_split(const FewArgs& a, bool i8) { return stream_steps(a.H * (i8 ? 1 : 2)) < kUpOwn ? 1 : kUpWaves; }

// Workgroups of gate/up, each with COLS columns of F.
int64_t up_groups(const FewArgs& a, int COLS) { return a.groups * ((a.F + COLS - 1) / COLS) + (a.Fs + COLS - 1) / COLS; }

template <bool I8, int RTM, int KS, bool HELD>
bool launch_up(const FewArgs& a, hipStream_t strm) {
  constexpr int COLS = 16 * kUpWaves / KS;
  constexpr auto k = k_few_gate_up<I8, RTM, KS, HELD>;
  const int lds = (RTM == 1 ? route_work_bytes(a.T * a.K, a.E, a.groups) : 0) +
                  (HELD ? kUpWaves * kHeldUpDepth * kSlot<2, 0, 0> + a.T * held_pitch(a.H) + kHeldTokens * (4 + 4 * kUpWaves)
                        : kUpWaves * kUpRing<RTM>);
  if (!lds_allowed<k>(lds)) return false;
  hipLaunchKernelGGL(k, dim3((unsigned)up_groups(a, COLS)), dim3(kUpWaves * kWave), lds, strm, a);
  return launch_status() == MOE_OK;
}

template <bool I8, int CT, bool HELD>
bool launch_down_as(const FewArgs& a, hipStream_t strm) {
  constexpr auto k = k_few_down<I8, CT, HELD>;
  const int S = a.T * a.K, ring = HELD ? kHeldDownDepth * kSlot<CT, 0, 0> : kDownRing;
  const int lds = route_bytes(S, a.groups) + kDownWaves * (ring + a.T * 16 * CT * 4) +
                  (HELD ? (S + a.T + 3) / 4 * 16 + held_h_bytes(S, a.T, a.F, a.Fs) : 0);
  if (!lds_allowed<k>(lds)) return false;
  hipLaunchKernelGGL(k, dim3((unsigned)((a.H + 16 * CT - 1) / (16 * CT))), dim3(kDownWaves * kWave), lds, strm, a);
  return launch_status() == MOE_OK;
}

// 16 columns for a workgroup while those workgroups do not exceed the 256 CUs, else 32:
// H = 1536 with 2 tokens 26.5 against 30.1 us for the layer, H = 4096 with 16 158 against 174;
// H = 5120 with 4 tokens 201 against 186, H = 7168 with 13 equal (int8 3 us slower with 16).
// Sixteen or four waves: within 2% of eight, H = 1536 more than 10% slower.
template <bool I8, bool HELD>
bool launch_down(const FewArgs& a, hipStream_t strm) {
  return a.H <= 16 * 256 ? launch_down_as<I8, 1, HELD>(a, strm) : launch_down_as<I8, 2, HELD>(a, strm);
}

template <bool I8, int RTM, int KS>
bool launch_y(const FewArgs& a, hipStream_t strm) {
  constexpr int COLS = 16 * kYCT<KS> * kYWaves / KS, lds = kYWaves * kYRing<I8, RTM, KS>;
  constexpr auto k = k_few_down_y<I8, RTM, KS>;
  const int64_t n = (a.groups + (a.Fs > 0)) * ((a.H + COLS - 1) / COLS);
  if (!lds_allowed<k>(lds)) return false;
  hipLaunchKernelGGL(k, dim3((unsigned)n), dim3(kYWaves * kWave), lds, strm, a);
  if (launch_status() != MOE_OK) return false;
  const dim3 grid((unsigned)((a.H + 1023) / 1024), (unsigned)a.T);
  if (a.K <= 8) hipLaunchKernelGGL(k_few_join<8>, grid, dim3(256), 0, strm, a);
  else hipLaunchKernelGGL(k_few_join<16>, grid, dim3(256), 0, strm, a);
  return launch_status() == MOE_OK;
}

// (no kernel is launched behind one that was not)
template <bool I8, int RTM>
moe_status few_launch(FewArgs& a, hipStream_t strm) {
  constexpr int ES = I8 ? 1 : 2;
  constexpr bool ROUTE = RTM > 1;
  const int S = a.T * a.K;
  if constexpr (I8 && RTM == 1) {
    if (few_held(a, true))
      return launch_up<true, 1, kUpWaves, true>(a, strm) && launch_down<true, true>(a, strm) ? MOE_OK : MOE_ERR_HIP;
  }
  if (ROUTE || I8) {
    hipLaunchKernelGGL((k_few_prep<ROUTE, I8>), dim3((ROUTE ? 1 : 0) + (I8 ? a.T + (a.smooth ? S : 0) : 0)), dim3(256),
                       ROUTE ? route_work_bytes(S, a.E, a.groups) : 16, strm, a);
    if (launch_status() != MOE_OK) return MOE_ERR_HIP;
  }
  if (!(up_split(a, I8) == 1 ? launch_up<I8, RTM, 1, false>(a, strm) : launch_up<I8, RTM, kUpWaves, false>(a, strm)))
    return MOE_ERR_HIP;
  if constexpr (I8) {
    // waves for a row to fit their registers (F = 14336: 3 us less of 165 to 278)
    const dim3 rows(S + (a.Fs ? a.T : 0));
    if (a.F > 8192 || a.Fs > 8192) hipLaunchKernelGGL(k_few_quant_h<8>, rows, dim3(8 * kWave), 0, strm, a);
    else hipLaunchKernelGGL(k_few_quant_h<4>, rows, dim3(4 * kWave), 0, strm, a);
    if (launch_status() != MOE_OK) return MOE_ERR_HIP;
  }
  bool ok;
  if (RTM == 1 && few_joins(a, I8))
    ok = launch_down<I8, false>(a, strm);
  else
    ok = stream_steps(a.F * ES) < kYOwn ? launch_y<I8, RTM, 1>(a, strm) : launch_y<I8, RTM, kYWaves>(a, strm);
  return ok ? MOE_OK : MOE_ERR_HIP;
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
  if (misaligned({x, w[0].codes, w[1].codes, w[2].codes, sw[0].codes, sw[1].codes, sw[2].codes, smooth,
                  workspace}))
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
  // gate/up's grid holds fewer than 2^32 threads on its axis (the others are smaller)
  if (up_groups(a, 16 * kUpWaves / up_split(a, i8)) * (kUpWaves * kWave) >= (int64_t)1 << 32) return MOE_ERR_UNSUPPORTED;
  if (S == 0) {
    // the error flag alone
    hipLaunchKernelGGL((k_few_prep<true, false>), dim3(1), dim3(256), route_work_bytes(0, a.E, 0), strm, a);
    return launch_status();
  }
  if (i8)
    return a.T <= 16 ? few_launch<true, 1>(a, strm) : (a.T <= 32 ? few_launch<true, 2>(a, strm) : few_launch<true, 4>(a, strm));
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
  a.T = (int)s->T; a.K = s->K; a.E = s->num_experts; a.H = s->H; a.F = s->F; a.Fs = shared_F;
  a.groups = a.T * a.K < s->num_experts ? a.T * a.K : s->num_experts;
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
