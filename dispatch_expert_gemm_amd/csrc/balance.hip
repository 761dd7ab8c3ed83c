// Balance loss and z loss of the router, per-expert counts, and their gradient to
// the logits (formulas at moe_balance_fwd in moe.h).
//
// Forward: the tokens of a sequence are cut into items of C tokens; a workgroup
// takes an item, reads each logit once, and leaves the item's column sums of
// softmax(logits), its histogram of the choices (LDS integer atomics), its sum of
// lse^2 and its number of active tokens in the workspace.  A second kernel sums
// the items of every sequence 64 columns at a time in 64 bits, and the last of
// its workgroups (a ticket that the first kernel clears) joins the sequences.
// No floating-point atomics; every sum has a fixed order.
//
// A token is held by GW lanes with Q runs of four consecutive logits each, so a
// wave holds 64/GW tokens and a row is read with 16-byte loads; sequence
// s owns item slots from off[s]/C + s, a bound that the host knows without the
// offsets: T/C + S slots.
//
// Backward: a workgroup takes a run of tokens, recomputes the softmax from the
// logits (read once) and writes each gradient once; the counts of a token's
// sequence stay in registers while the sequence stays the same.
#include "balance.hpp"
#include "common.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int64_t kMaxIds = 4096, kMaxSeqs = 1 << 20;

// Lane permutations within 16 lanes: xor 1, xor 2, then mirrors of 8 and of 16
// lanes, which reach the other half once the halves hold one value each.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

template <int GW, typename Op>
__device__ __forceinline__ float group_all(float v, Op op) {
  if constexpr (GW >= 2) v = op(v, dpp<0xB1>(v));
  if constexpr (GW >= 4) v = op(v, dpp<0x4E>(v));
  if constexpr (GW >= 8) v = op(v, dpp<0x141>(v));
  if constexpr (GW >= 16) v = op(v, dpp<0x140>(v));
  if constexpr (GW >= 32) v = op(v, __shfl_xor(v, 16, kWave));
  if constexpr (GW >= 64) v = op(v, __shfl_xor(v, 32, kWave));
  return v;
}
template <int GW>
__device__ __forceinline__ float group_max(float v) {
  return group_all<GW>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int GW>
__device__ __forceinline__ float group_sum(float v) {
  return group_all<GW>(v, [](float a, float b) { return a + b; });
}
// The sum of two whole numbers held as a float's bits.
__device__ __forceinline__ float add_bits(float a, float b) {
  return __int_as_float(__float_as_int(a) + __float_as_int(b));
}

struct BalanceArgs {
  const void* logits;
  const int32_t* idx;
  const uint8_t* mask;
  const int32_t* off;  // S + 1, or NULL: one sequence of all tokens
  int64_t T, slots;    // tokens; item slots
  int n, K, S, mask_ndim, C;
  int pitch;  // of psum's and hist's rows: n up to a multiple of 4
  // forward: per item
  float* psum;     // slots x pitch
  int32_t* hist;   // slots x pitch
  float* zsum;     // slots
  int32_t* ntok;   // slots
  double* dots;    // S x column blocks
  double* zseq;    // S
  uint32_t* ticket;
  float* loss;
  float* z_loss;
  int32_t* counts;      // S x n
  int32_t* counts2;     // the same, or NULL
  int32_t* seq_tokens;  // S, then their sum
  // backward
  const float* g_loss;
  const float* g_z;
  void* grad;
};

// Offsets are data: clamped to [0, T], so whatever they hold stays in bounds.
__device__ __forceinline__ int64_t off_at(const BalanceArgs& a, int s) {
  if (!a.off) return s ? a.T : 0;
  const int64_t o = a.off[s];
  return o < 0 ? 0 : (o > a.T ? a.T : o);
}

// The largest s of [0, S) with key(s) <= x, or 0: 64 probes of the range at a time.
template <typename Key>
__device__ __forceinline__ int find_last(int S, int64_t x, Key key) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = S;
  while (len > 1) {
    const int step = (len + 63) >> 6;
    const int s = lo + lane * step;
    const uint64_t m = __ballot(lane * step < len && key(s) <= x);
    const int last = m ? 63 - __clzll(m) : 0;
    const int left = len - last * step;
    lo += last * step;
    len = left < step ? left : step;
  }
  return lo;
}

// Four logits as they lie in memory: converted when they are used, so that a load a
// step ahead is not waited for.
template <typename In>
struct Raw4 {
  uint32_t w[sizeof(In)];  // four of fp32, or two of two bf16
};

// The four logits of row t from column c on; -inf past n.  VEC: n is a multiple of 4
// and the rows are aligned; otherwise the four begin anywhere, and a row's last ones
// are read one by one.
template <typename In, bool VEC>
__device__ __forceinline__ void load4(const BalanceArgs& a, int64_t t, int c, Raw4<In>& v) {
  const In* p = static_cast<const In*>(a.logits) + t * a.n + c;
#pragma unroll
  for (int j = 0; j < (int)sizeof(In); ++j) v.w[j] = sizeof(In) == 4 ? 0xff800000u : 0xff80ff80u;
  if (VEC ? c < a.n : c + 4 <= a.n) {
    if constexpr (!VEC) __builtin_memcpy(v.w, p, sizeof(v.w));
    else if constexpr (sizeof(In) == 4) *reinterpret_cast<uint4*>(v.w) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(v.w) = *reinterpret_cast<const uint2*>(p);
  } else if (!VEC && c < a.n) {
    const int left = a.n - c;  // 1 to 3
    if constexpr (sizeof(In) == 4) {
      v.w[0] = reinterpret_cast<const uint32_t*>(p)[0];
      if (left > 1) v.w[1] = reinterpret_cast<const uint32_t*>(p)[1];
      if (left > 2) v.w[2] = reinterpret_cast<const uint32_t*>(p)[2];
    } else {
      const bf16_t* q = reinterpret_cast<const bf16_t*>(p);
      v.w[0] = q[0] | (left > 1 ? (uint32_t)q[1] : 0xff80u) << 16;
      if (left > 2) v.w[1] = q[2] | 0xff800000u;
    }
  }
}

// A lane's part of row t (-inf where t >= t1): issued a step ahead of its use.  Rows of
// more than 1024 columns are held by a workgroup's 256 lanes (GW 256).
template <typename In, bool VEC, int GW, int Q>
__device__ __forceinline__ void load_row(const BalanceArgs& a, int64_t t, int64_t t1, Raw4<In> (&v)[Q]) {
  const int l = threadIdx.x & (GW - 1);
#pragma unroll
  for (int q = 0; q < Q; ++q) load4<In, VEC>(a, t, t < t1 ? (q * GW + l) * 4 : a.n, v[q]);
}

// The values of a row, a NaN read as -inf (fmaxf drops it).
template <typename In, int Q>
__device__ __forceinline__ void take_row(const Raw4<In> (&raw)[Q], float (&v)[Q][4]) {
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = sizeof(In) == 4 ? raw[q].w[j % sizeof(In)]
                                         : (j & 1 ? raw[q].w[j / 2 % sizeof(In)] & 0xffff0000u
                                                  : raw[q].w[j / 2 % sizeof(In)] << 16);
      v[q][j] = fmaxf(__uint_as_float(b), -INFINITY);
    }
}

// exp(v - m) in place of the row's logits (__expf: |v - m| 2^-24 from the product with
// log2(e) and two units in the last place, of the size of the sum's own rounding); m the row's largest (`top` over its lanes),
// total the sum (`sum`).  A row that holds nothing above -inf gives zeros and total 0.
template <int Q, typename Top, typename Sum>
__device__ __forceinline__ void row_exp(float (&v)[Q][4], float& m, float& total, Top top, Sum sum) {
  m = -INFINITY;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, v[q][j]);
  m = top(m);
  const float base = m != -INFINITY ? m : 0.f;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[q][j] = __expf(v[q][j] - base);
      s += v[q][j];
    }
  total = sum(s);
}

// A value over a workgroup's 256 lanes: its waves meet in one of two rows of LDS in
// turn, so one barrier a value is enough (a row is written again only behind the
// barrier of the value between).
struct Meet {
  float (*rows)[kWaves];
  int turn;
  template <typename Op>
  __device__ __forceinline__ float all(float v, Op op) {
    v = group_all<kWave>(v, op);
    float* r = rows[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
    __syncthreads();
    v = r[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v = op(v, r[w]);
    return v;
  }
  __device__ __forceinline__ float max(float v) {
    return all(v, [](float a, float b) { return fmaxf(a, b); });
  }
  __device__ __forceinline__ float sum(float v) {
    return all(v, [](float a, float b) { return a + b; });
  }
};

// A lane's part of token t's mask (0 where t is not in [lo, hi)), as it lies in
// memory: loaded with the token's row, looked at with it.  Four or eight lanes hold up to 16
// slots, more lanes one each.
template <int GW>
__device__ __forceinline__ uint32_t load_mask(const BalanceArgs& a, int64_t t, int64_t lo, int64_t hi) {
  if (t < lo || t >= hi) return 0u;
  if (a.mask_ndim == 0) return 1u;
  if (a.mask_ndim == 1) return a.mask[t];
  const int l = threadIdx.x & (GW - 1);
  uint32_t m = l < a.K ? a.mask[t * a.K + l] : 0u;
  if constexpr (GW < 16)
    for (int k = l + GW; k < a.K; k += GW) m |= a.mask[t * a.K + k];
  return m;
}

// Whether the token whose lanes hold these parts counts.
template <int GW>
__device__ __forceinline__ bool token_on(uint32_t mask) {
  const int lane = threadIdx.x & 63;
  const uint64_t b = __ballot(mask != 0);
  if constexpr (GW == 64) return b != 0;
  else return ((b >> (lane & ~(GW - 1))) & ((1ull << GW) - 1)) != 0;
}

template <int W>
__device__ __forceinline__ double block_sum(double v, double* red) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  __syncthreads();
  if ((tid & 63) == 0) red[tid >> 6] = v;
  __syncthreads();
  double r = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) r += red[w];
  return r;
}

// Waves of a workgroup of items: a wave waits for its tokens' rows, so eight (32768
// tokens of 1024 columns, the gradient left in the caches: 4 waves 67 us, 8 waves and
// rows loaded ahead 43; rows loaded two steps ahead gain nothing).  The only workgroup of a small batch takes 16.
template <bool ALONE>
constexpr int kItemWaves = ALONE ? 16 : 8;
constexpr int kSumRows = 4;  // rows of column sums in LDS that the waves are added into

// The tokens of an item, from the offsets; false where no sequence fills the slot.
__device__ __forceinline__ bool tokens_of(const BalanceArgs& a, int64_t item, int64_t& t0, int64_t& t1) {
  int s = 0;
  if (a.off) s = find_last(a.S, item, [&](int i) { return off_at(a, i) / a.C + i; });
  const int64_t lo = off_at(a, s), hi = off_at(a, s + 1);
  t0 = lo + (item - (lo / a.C + s)) * a.C;
  t1 = t0 + a.C < hi ? t0 + a.C : hi;
  return t0 >= lo && t0 < t1;
}

// The choices of tokens t0 to t1 into the histogram, a thread each: with each token's
// among its logits the wave would wait for them too.
__device__ __forceinline__ void count_choices(const BalanceArgs& a, int64_t t0, int64_t t1, int* hist) {
  const int slots = (int)(t1 - t0) * a.K;
  for (int i = threadIdx.x; i < slots; i += blockDim.x) {
    const int64_t at = t0 * a.K + i;
    const int32_t e = a.idx[at];
    bool on = (uint32_t)e < (uint32_t)a.n;
    if (a.mask_ndim) on = on && a.mask[a.mask_ndim == 2 ? at : t0 + (uint32_t)i / (uint32_t)a.K];
    if (on) atomicAdd(&hist[e], 1);
  }
}

// ALONE: the batch is one item, so this workgroup finishes it.
template <typename In, bool VEC, int GW, int Q, bool ALONE>
__global__ __launch_bounds__(kWave * kItemWaves<ALONE>, ALONE ? 1 : 4) void k_balance_items(BalanceArgs a) {
  constexpr int W = kItemWaves<ALONE>, RW = kSumRows, G = kWave / GW;
  extern __shared__ float smem[];
  float* rows = smem;                                   // RW x n column sums
  int* hist = reinterpret_cast<int*>(smem + RW * a.n);  // n
  __shared__ float zs[W];
  __shared__ int ns[W];
  __shared__ double red[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & (GW - 1);
  const int64_t item = blockIdx.x;
  if (!ALONE && item == 0 && tid == 0) *a.ticket = 0;
  int64_t t0 = 0, t1 = a.T;
  if (!ALONE && !tokens_of(a, item, t0, t1)) return;  // (never read)
  for (int i = tid; i < a.n; i += kWave * W) hist[i] = 0;
  float v[Q][4];
  Raw4<In> next[Q];
  load_row<In, VEC, GW, Q>(a, t0 + wave * G + lane / GW, t1, next);
  uint32_t mask_next = load_mask<GW>(a, t0 + wave * G + lane / GW, t0, t1);
  __syncthreads();
  count_choices(a, t0, t1, hist);
  float p[Q][4];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) p[q][j] = 0.f;
  float z = 0.f;
  int nt = 0;
  for (int64_t b = t0 + wave * G; b < t1; b += W * G) {
    const int64_t t = b + lane / GW;
    take_row<In, Q>(next, v);
    const bool on = token_on<GW>(mask_next);
    load_row<In, VEC, GW, Q>(a, t + W * G, t1, next);
    mask_next = load_mask<GW>(a, t + W * G, t0, t1);
    float m, total;
    row_exp(v, m, total, group_max<GW>, group_sum<GW>);
    const float inv = on && total != 0.f ? 1.0f / total : 0.f;
    if (on) {  // (a token that is off adds nothing, not even a NaN)
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[q][j] += v[q][j] * inv;
      const float lse = total != 0.f ? m + __logf(total) : 0.f;
      z += lse * lse;
      ++nt;
    }
  }
  // the wave's tokens, then the workgroup's waves in order
#pragma unroll
  for (int o = GW; o < kWave; o <<= 1) {
    z += __shfl_xor(z, o, kWave);
    nt += __shfl_xor(nt, o, kWave);
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) p[q][j] += __shfl_xor(p[q][j], o, kWave);
  }
  if (lane == 0) {
    zs[wave] = z;
    ns[wave] = nt;
  }
#pragma unroll
  for (int w = 0; w < W / RW; ++w) {
    if (wave / RW == w && lane < GW) {
      float* row = rows + (wave % RW) * a.n;
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = (q * GW + l) * 4 + j;
          if (c < a.n) row[c] = w ? row[c] + p[q][j] : p[q][j];
        }
    }
    __syncthreads();
  }
  double dot = 0;
  for (int c = tid; c < a.n; c += kWave * W) {
    float v = rows[c];
#pragma unroll
    for (int r = 1; r < RW; ++r) v += rows[r * a.n + c];
    if constexpr (ALONE) {
      a.counts[c] = hist[c];
      if (a.counts2) a.counts2[c] = hist[c];
      dot += (double)v * hist[c];
    } else {
      a.psum[item * a.pitch + c] = v;
      a.hist[item * a.pitch + c] = hist[c];
    }
  }
  if constexpr (ALONE) dot = block_sum<W>(dot, red);
  if (tid == 0) {
    double v = 0;
    int k = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      v += zs[w];
      k += ns[w];
    }
    if constexpr (ALONE) {
      a.seq_tokens[0] = a.seq_tokens[1] = k;
      *a.loss = k ? (float)(dot * a.n / ((double)a.K * k * k)) : 0.f;
      *a.z_loss = k ? (float)(v / k) : 0.f;
    } else {
      a.zsum[item] = (float)v;
      a.ntok[item] = k;
    }
  }
}

// Rows of more than 1024 columns: the workgroup's 256 lanes hold a token, Q runs each,
// so a lane keeps the sums of its own columns and a CU holds eight tokens (a wave for
// a token takes 200 to 256 registers: 8192 x 4096 89 us forward and 166 backward, 45 and
// 53 so).
template <typename In, bool VEC, int Q>
__global__ __launch_bounds__(kThreads) void k_balance_items_wide(BalanceArgs a) {
  extern __shared__ float smem[];
  int* hist = reinterpret_cast<int*>(smem);  // n
  __shared__ float rows[2][kWaves];
  const int tid = threadIdx.x;
  const int64_t item = blockIdx.x;
  if (item == 0 && tid == 0) *a.ticket = 0;
  int64_t t0, t1;
  if (!tokens_of(a, item, t0, t1)) return;  // (never read)
  for (int i = tid; i < a.n; i += kThreads) hist[i] = 0;
  Meet meet{rows, 0};
  float v[Q][4], p[Q][4];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) p[q][j] = 0.f;
  Raw4<In> next[Q];
  load_row<In, VEC, kThreads, Q>(a, t0, t1, next);
  uint32_t mask_next = load_mask<kWave>(a, t0, t0, t1);
  __syncthreads();
  count_choices(a, t0, t1, hist);
  float z = 0.f;
  int nt = 0;
  for (int64_t t = t0; t < t1; ++t) {
    take_row<In, Q>(next, v);
    const bool on = token_on<kWave>(mask_next);
    load_row<In, VEC, kThreads, Q>(a, t + 1, t1, next);
    mask_next = load_mask<kWave>(a, t + 1, t0, t1);
    float m, total;
    row_exp(v, m, total, [&](float x) { return meet.max(x); }, [&](float x) { return meet.sum(x); });
    if (on) {
      const float inv = total != 0.f ? 1.0f / total : 0.f;
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[q][j] += v[q][j] * inv;
      const float lse = total != 0.f ? m + __logf(total) : 0.f;
      z += lse * lse;
      ++nt;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int c = (q * kThreads + tid) * 4;
    if (c < a.n)
      *reinterpret_cast<float4*>(a.psum + item * a.pitch + c) = make_float4(p[q][0], p[q][1], p[q][2], p[q][3]);
  }
  for (int c = tid; c < a.n; c += kThreads) a.hist[item * a.pitch + c] = hist[c];
  if (tid == 0) {
    a.zsum[item] = z;
    a.ntok[item] = nt;
  }
}

// Sums of three values over a workgroup's waves, in every lane of the first.
template <int W>
__device__ __forceinline__ void block_sum3(double& x, double& y, double& z, double (*red)[3]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    x += __shfl_xor(x, o, kWave);
    y += __shfl_xor(y, o, kWave);
    z += __shfl_xor(z, o, kWave);
  }
  if (lane == 0) {
    red[wave][0] = x;
    red[wave][1] = y;
    red[wave][2] = z;
  }
  __syncthreads();
  x = y = z = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    x += red[w][0];
    y += red[w][1];
    z += red[w][2];
  }
}

template <typename T>
__device__ __forceinline__ void put(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get(T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One workgroup for a sequence and 64 columns: 16 lanes hold four columns each, and
// the 64 groups of them share the sequence's items, eight loads in flight.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(kWave * kJoinWaves) void k_balance_join(BalanceArgs a) {
  constexpr int W = kJoinWaves, kRows = W * 4;
  __shared__ double dsum[W][kWave];
  __shared__ int csum[W][kWave];
  __shared__ double red[W][3];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int blocks = (a.n + 63) / 64;
  const int s = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const int64_t lo = off_at(a, s), hi = off_at(a, s + 1);
  const int64_t i0 = lo / a.C + s;
  int64_t i1 = hi > lo ? i0 + (hi - lo + a.C - 1) / a.C : i0;
  if (i1 > a.slots) i1 = a.slots;
  double p[4] = {0, 0, 0, 0}, z = 0, nt = 0;
  int k[4] = {0, 0, 0, 0};
  const int c4 = cb * 64 + (lane & 15) * 4;
  if (c4 < a.n)
#pragma unroll 4
    for (int64_t i = i0 + wave * 4 + (lane >> 4); i < i1; i += kRows) {
      const float4 f = *reinterpret_cast<const float4*>(a.psum + i * a.pitch + c4);
      const int4 h = *reinterpret_cast<const int4*>(a.hist + i * a.pitch + c4);
      p[0] += f.x; p[1] += f.y; p[2] += f.z; p[3] += f.w;
      k[0] += h.x; k[1] += h.y; k[2] += h.z; k[3] += h.w;
    }
  if (cb == 0 && wave == 0)
#pragma unroll 4
    for (int64_t i = i0 + lane; i < i1; i += kWave) {
      z += a.zsum[i];
      nt += a.ntok[i];
    }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int o = 16; o < kWave; o <<= 1) {
      p[j] += __shfl_xor(p[j], o, kWave);
      k[j] += __shfl_xor(k[j], o, kWave);
    }
    if (lane < 16) {
      dsum[wave][lane * 4 + j] = p[j];
      csum[wave][lane * 4 + j] = k[j];
    }
  }
  __syncthreads();
  double dot = 0;
  if (wave == 0) {
    const int c = cb * 64 + lane;
    if (c < a.n) {
      double ps = 0;
      int ks = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        ps += dsum[w][lane];
        ks += csum[w][lane];
      }
      a.counts[(int64_t)s * a.n + c] = ks;
      if (a.counts2) a.counts2[(int64_t)s * a.n + c] = ks;
      dot = ps * ks;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      dot += __shfl_xor(dot, o, kWave);
      z += __shfl_xor(z, o, kWave);
      nt += __shfl_xor(nt, o, kWave);
    }
  }
  if (gridDim.x == 1) {
    if (tid == 0) {
      a.seq_tokens[0] = a.seq_tokens[1] = (int32_t)nt;
      *a.loss = nt > 0 ? (float)(dot * a.n / (a.K * nt * nt)) : 0.f;
      *a.z_loss = nt > 0 ? (float)(z / nt) : 0.f;
    }
    return;
  }
  // What the last workgroup reads goes to memory and back as device-scope atomics,
  // which no L2 holds back, waited for before the ticket: a fence would write back and
  // drop whole L2s (13 us for this kernel in place of 8).
  if (tid == 0) {
    put(&a.dots[blockIdx.x], dot);
    if (cb == 0) {
      put(&a.zseq[s], z);
      put(&a.seq_tokens[s], (int32_t)nt);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  double N = 0, loss = 0;
  z = 0;
  for (int i = tid; i < a.S; i += kWave * W) {
    const int m = get(&a.seq_tokens[i]);
    double d = 0;
#pragma unroll 4
    for (int b = 0; b < blocks; ++b) d += get(&a.dots[(int64_t)i * blocks + b]);
    if (m > 0) loss += d / m;
    N += m;
    z += get(&a.zseq[i]);
  }
  block_sum3<W>(N, loss, z, red);
  if (tid == 0) {
    a.seq_tokens[a.S] = (int32_t)N;
    *a.loss = N > 0 ? (float)(loss * a.n / (a.K * N)) : 0.f;
    *a.z_loss = N > 0 ? (float)(z / N) : 0.f;
  }
}

template <typename In, bool VEC, bool PAST>
__device__ __forceinline__ void store4(const BalanceArgs& a, int64_t t, int c, const float* v) {
  In* p = static_cast<In*>(a.grad) + t * a.n + c;
  if (VEC ? c < a.n : c + 4 <= a.n) {
    if constexpr (sizeof(In) == 4) {
      typedef float f32x4_t __attribute__((ext_vector_type(4)));
      const f32x4_t r = {v[0], v[1], v[2], v[3]};
      if constexpr (PAST) __builtin_nontemporal_store(r, reinterpret_cast<f32x4_t*>(p));
      else if constexpr (VEC) *reinterpret_cast<f32x4_t*>(p) = r;
      else __builtin_memcpy(p, &r, 16);
    } else {
      const uint2 r = make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
      if constexpr (VEC) *reinterpret_cast<uint2*>(p) = r;
      else __builtin_memcpy(p, &r, 8);
    }
  } else if (!VEC && c < a.n) {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (c + j < a.n) {
        if constexpr (sizeof(In) == 4) p[j] = v[j];
        else reinterpret_cast<bf16_t*>(p)[j] = (bf16_t)f2bf(v[j]);
      }
  }
}

// PAST: the gradient does not fit the caches and is written around them.  GW 256: the
// workgroup holds one token.
template <typename In, bool VEC, int GW, int Q, bool PAST>
__global__ __launch_bounds__(kThreads) void k_balance_bwd(BalanceArgs a) {
  constexpr bool kWide = GW > kWave;
  constexpr int kMaskLanes = kWide ? kWave : GW, kStep = kThreads / GW;
  __shared__ float rows[2][kWaves];
  Meet meet{rows, 0};
  const int tid = threadIdx.x, l = tid & (GW - 1);
  auto sum = [&](float x) {
    if constexpr (kWide) return meet.sum(x);
    else return group_sum<GW>(x);
  };
  auto top = [&](float x) {
    if constexpr (kWide) return meet.max(x);
    else return group_max<GW>(x);
  };
  const int64_t t0 = (int64_t)blockIdx.x * a.C;
  const int64_t t1 = t0 + a.C < a.T ? t0 + a.C : a.T;
  // (every load before the first use of one: a small batch waits for memory once)
  float v[Q][4];
  Raw4<In> next[Q];
  load_row<In, VEC, GW, Q>(a, t0 + tid / GW, t1, next);
  uint32_t mask_next = load_mask<kMaskLanes>(a, t0 + tid / GW, t0, t1);
  // the last sequence that begins at or before the run's first token
  int s = a.off ? find_last(a.S, t0, [&](int i) { return off_at(a, i); }) : 0;
  int64_t s0 = off_at(a, s), s1 = off_at(a, s + 1);
  // The counts are used less their mean (a whole number): as sum_j p_j = 1, that leaves
  // c - sum_j p_j c_j as it is, but its rounding then goes by the counts' differences.  Near an
  // even load the counts are large beside them (65536 x 64, top 8, two counts one off the mean:
  // the gradient 0.8% off with the counts themselves, 1e-7 so).
  int held = s, tokens, c[Q][4];
  bool centred = false;
  auto hold = [&]() {
    centred = false;
    tokens = a.seq_tokens[s];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = (q * GW + l) * 4 + j;
        c[q][j] = e < a.n ? a.counts[(int64_t)s * a.n + e] : 0;
      }
  };
  auto centre = [&]() {  // at the first use, so that a row's work covers the counts' loads
    centred = true;
    int part = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) part += c[q][j];
    float bits = __int_as_float(part);
    if constexpr (kWide) bits = meet.all(bits, add_bits);
    else bits = group_all<GW>(bits, add_bits);
    const int mean = __float_as_int(bits) / a.n;  // (exact for equal counts of any size)
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[q][j] = (q * GW + l) * 4 + j < a.n ? c[q][j] - mean : 0;
  };
  hold();
  const int all = a.seq_tokens[a.S];
  const float g_loss = a.g_loss ? *a.g_loss : 0.f, g_z = a.g_z ? *a.g_z : 0.f;
  const float gb = (float)((double)g_loss * a.n / ((double)a.K * all)), gz = (float)(g_z * 2.0 / all);
  for (int64_t b = t0; b < t1; b += kStep) {  // (the whole workgroup)
    const int64_t t = b + tid / GW;
    const bool in = t < t1;
    take_row<In, Q>(next, v);
    const bool unmasked = token_on<kMaskLanes>(mask_next);
    load_row<In, VEC, GW, Q>(a, t + kStep, t1, next);
    mask_next = load_mask<kMaskLanes>(a, t + kStep, t0, t1);
    if (in && t >= s1 && s + 1 < a.S) {  // the next sequence, or behind it the last that begins at or before t
      s0 = s1;
      s1 = off_at(a, ++s + 1);
      if (t >= s1 && s + 1 < a.S) {
        // (halving: empty sequences, offsets padded to a number of sequences, may be any many;
        // 70 tokens among 131072 sequences 14 ms one by one, 9 us so)
        int lo = s + 1, end = a.S;
        while (end - lo > 1) {
          const int mid = lo + (end - lo) / 2;
          if (off_at(a, mid) <= t) lo = mid;
          else end = mid;
        }
        s = lo;
        s0 = off_at(a, s);
        s1 = off_at(a, s + 1);
      }
    }
    const bool on = unmasked && in && t >= s0 && t < s1;
    if (on && held != s) {
      held = s;
      hold();
    }
    float m, total;
    row_exp(v, m, total, top, sum);
    if (!centred) centre();  // (the lanes of a token together)
    const bool some = on && total != 0.f;
    const float inv = some ? 1.0f / total : 0.f;
    const float share = some ? gb / (float)tokens : 0.f;
    float d = 0.f;
    if (some)
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[q][j] *= inv;
          d += v[q][j] * (float)c[q][j];
        }
    d = sum(d);
    const float zt = some ? gz * (m + __logf(total)) : 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = some ? v[q][j] * (share * ((float)c[q][j] - d) + zt) : 0.f;
      if (in) store4<In, VEC, PAST>(a, t, (q * GW + l) * 4, r);
    }
  }
}

// Lanes of a token.  The more runs of four a lane holds, the fewer steps the sum over
// the lanes takes and the more tokens share a wave's instructions (65536 tokens,
// forward + backward in us: 260 columns fp32 64 lanes 34 + 31, 32 lanes 28 + 26; 128
// bf16 32 lanes 20 + 15, 16 lanes 18 + 14), until a small batch has too few items (8192
// tokens of 64 columns 16 lanes 8.8, 8 lanes 9.6) or the registers end (32768 x 1024 by 32
// lanes 159 + 55 for 40 + 52).
inline int group_lanes(int64_t n) {
  return n <= 16 ? 4 : (n <= 32 ? 8 : (n <= 128 ? 16 : (n <= 512 ? 32 : (n <= 1024 ? 64 : 256))));
}
// Tokens that a workgroup of `waves` takes at a time.
inline int step_tokens(int64_t n, int waves) { return waves * kWave / group_lanes(n); }

// Tokens of an item: whole steps, about 500 items of a batch: two workgroups of eight
// waves a CU, and few rows of sums to join (32768 x 1024, forward and backward: 500 items
// 89.7 us, 700 91.8, 1500 93.4).  Workgroups of four waves (wide rows): four a CU (32768 x
// 2048, the forward: 500 items 103 us, 1000 71, 2000 75), of four tokens or more.
inline int64_t item_tokens(int64_t T, int64_t n) {
  const int64_t step = n <= 1024 ? step_tokens(n, kItemWaves<false>) : kWaves;
  const int64_t items = n <= 1024 ? 500 : 1000, per = (T + items - 1) / items;
  return per ? (per + step - 1) / step * step : step;
}

// One workgroup does a small batch without sequences in one launch.  Forward in us by one
// launch and by two: 1 x 64 4.1 and 6.6, 256 x 64 6.8 and 6.9, 128 x 256 8.7 and 10.3, 32 x 1024
// 9.2 and 11.5.  A workgroup's time goes by its steps of tokens, of which narrow rows have more
// for the same logits: 512 x 64 9.9 and 7.0, 4096 x 8 15.8 and 7.6, 16384 x 2 58 and 8.3.
inline bool alone(int64_t T, int64_t n, int64_t num_seqs) { return num_seqs == 0 && n <= 1024 && T * n <= 32768; }

struct Layout {
  int64_t slots, psum, hist, zsum, ntok, dots, zseq, ticket, bytes;
};
Layout layout_of(int64_t T, int64_t n, int64_t S) {
  Layout w;
  w.slots = T / item_tokens(T, n) + S;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const int64_t pitch = (n + 3) / 4 * 4;
  w.psum = take(w.slots * pitch * 4);
  w.hist = take(w.slots * pitch * 4);
  w.zsum = take(w.slots * 4);
  w.ntok = take(w.slots * 4);
  w.dots = take(S * ((n + 63) / 64) * 8);
  w.zseq = take(S * 8);
  w.ticket = take(4);
  w.bytes = at;
  return w;
}

moe_status check_balance(int64_t T, int64_t n, int32_t K, int64_t S, int32_t mask_ndim, int32_t dtype) {
  if (T < 0 || T > 0x7fffffff || n < 1 || n > kMaxIds || K < 1 || K > 16 || K > n) return MOE_ERR_BAD_SHAPE;
  if (T * K > 0x7fffffff) return MOE_ERR_BAD_SHAPE;  // counts are int32
  if (S < 0 || S > kMaxSeqs) return MOE_ERR_BAD_SHAPE;
  if (mask_ndim < 0 || mask_ndim > 2) return MOE_ERR_BAD_RANGE;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP32) return MOE_ERR_BAD_RANGE;
  return MOE_OK;
}

// Calls f(In type tag, VEC, GW, Q) for n columns.
template <typename In, bool VEC, typename Fn>
void launch_gq(int64_t n, Fn f) {
  if (n <= 16) f.template operator()<In, VEC, 4, 1>();
  else if (n <= 32) f.template operator()<In, VEC, 8, 1>();
  else if (n <= 64) f.template operator()<In, VEC, 16, 1>();
  else if (n <= 128) f.template operator()<In, VEC, 16, 2>();
  else if (n <= 256) f.template operator()<In, VEC, 32, 2>();
  else if (n <= 384) f.template operator()<In, VEC, 32, 3>();
  else if (n <= 512) f.template operator()<In, VEC, 32, 4>();
  else if (n <= 1024) f.template operator()<In, VEC, 64, 4>();
  else if (n <= 2048) f.template operator()<In, VEC, 256, 2>();
  else f.template operator()<In, VEC, 256, 4>();
}

struct LaunchItems {
  const BalanceArgs& a;
  hipStream_t strm;
  bool one;
  template <typename In, bool VEC, int GW, int Q>
  void operator()() const {
    if constexpr (GW > kWave) {
      hipLaunchKernelGGL((k_balance_items_wide<In, VEC, Q>), dim3((unsigned)a.slots), dim3(kThreads), a.n * 4, strm, a);
    } else {
      const unsigned lds = (kSumRows + 1) * a.n * 4;
      if (one) hipLaunchKernelGGL((k_balance_items<In, VEC, GW, Q, true>), dim3(1), dim3(kWave * kItemWaves<true>), lds,
                                  strm, a);
      else hipLaunchKernelGGL((k_balance_items<In, VEC, GW, Q, false>), dim3((unsigned)a.slots),
                              dim3(kWave * kItemWaves<false>), lds, strm, a);
    }
  }
};
struct LaunchBwd {
  const BalanceArgs& a;
  hipStream_t strm;
  template <typename In, bool VEC, int GW, int Q>
  void operator()() const {
    const dim3 grid((unsigned)((a.T + a.C - 1) / a.C));
    // a gradient past the L2s' 32 MB that stayed in the caches would go to memory while
    // the next kernel reads (32768 x 1024 fp32, forward and backward 107 us, so 101)
    constexpr bool kWide = VEC && sizeof(In) == 4;
    if (kWide && a.T * a.n * 4 > (32 << 20))
      hipLaunchKernelGGL((k_balance_bwd<In, VEC, GW, Q, kWide>), grid, dim3(kThreads), 0, strm, a);
    else
      hipLaunchKernelGGL((k_balance_bwd<In, VEC, GW, Q, false>), grid, dim3(kThreads), 0, strm, a);
  }
};

template <typename Launch>
void launch_any(const BalanceArgs& a, int32_t dtype, bool vec, const Launch& f) {
  if (dtype == MOE_DTYPE_FP32) {
    if (vec) launch_gq<float, true>(a.n, f);
    else launch_gq<float, false>(a.n, f);
  } else {
    if (vec) launch_gq<bf16_t, true>(a.n, f);
    else launch_gq<bf16_t, false>(a.n, f);
  }
}

inline bool rows_aligned(const void* p, int64_t n, int32_t dtype) {
  return n % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (dtype == MOE_DTYPE_FP32 ? 16 : 8) == 0;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_balance_workspace_size(int64_t T, int64_t n_ids, int64_t num_seqs, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL_ARG;
  const moe_status st = check_balance(T, n_ids, 1, num_seqs, 0, MOE_DTYPE_FP32);
  if (st != MOE_OK) return st;
  *bytes = (size_t)layout_of(T, n_ids, num_seqs ? num_seqs : 1).bytes;
  return MOE_OK;
}

moe_status moe::balance_forward(int64_t T, int64_t n_ids, int32_t K, int64_t num_seqs, int32_t mask_ndim, int32_t dtype,
                                const void* logits, const int32_t* topk_idx, const uint8_t* x_active_mask,
                                const int32_t* seq_offsets, float* loss, float* z_loss, int32_t* counts,
                                int32_t* counts_again, int32_t* seq_tokens, void* workspace, size_t ws_bytes,
                                void* stream) {
  const moe_status st = check_balance(T, n_ids, K, num_seqs, mask_ndim, dtype);
  if (st != MOE_OK) return st;
  MOE_NEED(logits, T);
  MOE_NEED(topk_idx, T);
  if (mask_ndim) MOE_NEED(x_active_mask, T);
  if ((num_seqs && !seq_offsets) || !loss || !z_loss || !counts || !seq_tokens) return MOE_ERR_NULL_ARG;
  const int64_t S = num_seqs ? num_seqs : 1;
  const Layout w = layout_of(T, n_ids, S);
  if (!workspace || ws_bytes < (size_t)w.bytes) return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 16) return MOE_ERR_BAD_SHAPE;
  const int64_t blocks = S * ((n_ids + 63) / 64);
  if (w.slots > 0x3fffff || blocks > 0x3fffff) return MOE_ERR_BAD_SHAPE;  // 2^32 threads of a launch
  const bool one = alone(T, n_ids, num_seqs);
  char* ws = static_cast<char*>(workspace);
  BalanceArgs a{};
  a.logits = logits;
  a.idx = topk_idx;
  a.mask = x_active_mask;
  a.off = num_seqs ? seq_offsets : nullptr;
  a.T = T;
  a.slots = w.slots;
  a.n = (int)n_ids;
  a.K = K;
  a.S = (int)S;
  a.mask_ndim = mask_ndim;
  a.C = (int)item_tokens(T, n_ids);
  a.pitch = (int)((n_ids + 3) / 4 * 4);
  a.psum = reinterpret_cast<float*>(ws + w.psum);
  a.hist = reinterpret_cast<int32_t*>(ws + w.hist);
  a.zsum = reinterpret_cast<float*>(ws + w.zsum);
  a.ntok = reinterpret_cast<int32_t*>(ws + w.ntok);
  a.dots = reinterpret_cast<double*>(ws + w.dots);
  a.zseq = reinterpret_cast<double*>(ws + w.zseq);
  a.ticket = reinterpret_cast<uint32_t*>(ws + w.ticket);
  a.loss = loss;
  a.z_loss = z_loss;
  a.counts = counts;
  a.counts2 = counts_again;
  a.seq_tokens = seq_tokens;
  launch_any(a, dtype, rows_aligned(logits, n_ids, dtype), LaunchItems{a, as_stream(stream), one});
  const moe_status first = launch_status();
  if (first != MOE_OK || one) return first;
  hipLaunchKernelGGL(k_balance_join, dim3((unsigned)blocks), dim3(kWave * kJoinWaves), 0, as_stream(stream), a);
  return launch_status();
}

extern "C" moe_status moe_balance_fwd(int64_t T, int64_t n_ids, int32_t K, int64_t num_seqs, int32_t mask_ndim,
                                      int32_t dtype, const void* logits, const int32_t* topk_idx,
                                      const uint8_t* x_active_mask, const int32_t* seq_offsets, float* loss,
                                      float* z_loss, int32_t* counts, int32_t* seq_tokens, void* workspace,
                                      size_t ws_bytes, void* stream) {
  return balance_forward(T, n_ids, K, num_seqs, mask_ndim, dtype, logits, topk_idx, x_active_mask, seq_offsets, loss,
                         z_loss, counts, nullptr, seq_tokens, workspace, ws_bytes, stream);
}

extern "C" moe_status moe_balance_bwd(int64_t T, int64_t n_ids, int32_t K, int64_t num_seqs, int32_t mask_ndim,
                                      int32_t dtype, const void* logits, const uint8_t* x_active_mask,
                                      const int32_t* seq_offsets, const int32_t* counts, const int32_t* seq_tokens,
                                      const float* grad_loss, const float* grad_z_loss, void* grad_logits,
                                      void* stream) {
  const moe_status st = check_balance(T, n_ids, K, num_seqs, mask_ndim, dtype);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!logits || !counts || !seq_tokens || !grad_logits || (num_seqs && !seq_offsets) ||
      (mask_ndim && !x_active_mask))
    return MOE_ERR_NULL_ARG;
  BalanceArgs a{};
  a.logits = logits;
  a.mask = x_active_mask;
  a.off = num_seqs ? seq_offsets : nullptr;
  a.T = T;
  a.n = (int)n_ids;
  a.K = K;
  a.S = num_seqs ? (int)num_seqs : 1;
  a.mask_ndim = mask_ndim;
  // runs of tokens: enough workgroups for every CU, whole steps each
  const int64_t step = step_tokens(n_ids, kWaves), per = (T + 2047) / 2048;
  a.C = (int)((per + step - 1) / step * step);
  a.counts = const_cast<int32_t*>(counts);
  a.seq_tokens = const_cast<int32_t*>(seq_tokens);
  a.g_loss = grad_loss;
  a.g_z = grad_z_loss;
  a.grad = grad_logits;
  launch_any(a, dtype, rows_aligned(logits, n_ids, dtype) && rows_aligned(grad_logits, n_ids, dtype),
             LaunchBwd{a, as_stream(stream)});
  return launch_status();
}
