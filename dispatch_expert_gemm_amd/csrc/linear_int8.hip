// The matrix product on 8-bit integers with a scale for each token and each
// output channel, moe_linear_int8: out[m, n] = bf16((sum_k xq[m, k] wq[n, k]) *
// (xs[m] * ws[n]) + bias[n]), the sum exact in int32; and its dynamic form, which
// first quantises bf16 rows (int8_scale in stream_mfma.hpp).
//
// k_linear_rows: one workgroup per (16 CT output columns, up to 64 rows).  Its waves
// split the contraction, each streaming its part of the weight rows from
// memory into the matrix cores (stream_mfma.hpp); the int32 partial sums meet in
// LDS, where their order does not matter.  k_linear_held: the same for one or two bf16
// rows, quantised inside.  Bound: HBM, N * K bytes of weights, and for small ones the
// launch: one row of 7168 x 7168 11.0 us (4.7 TB/s; 10.7 for a call among others, which
// overlap), 37 rows of 7168 x 2048 6.6 us.
//
// k_linear_tiles: tiles of 64 x 128 to 256 x 256, both operands in LDS.  512 x 4096 x 7168
// takes 26.1 us (1.15 POP/s), on 256 tiles: about 7 are a workgroup's beginning and end, and
// the loop takes its operands at 72 bytes per ns and CU, where the row kernel reaches
// about 95.  Bound, for large products: power.  8192 x 14336 x 4096 takes 463 us where the
// clock stays at 1.93 GHz and up to 545 where it falls to 1.62; 382 of the 463 grow with K
// (2.52 POP/s there).  The matrix cores are busy for 51% of its cycles, 70% of those that
// grow with K.  On 128 x 256 tiles 530 us; four waves of 128 x 128, with two thirds of the LDS
// reads, take the same time.
#include <algorithm>
#include <type_traits>

#include "stream_mfma.hpp"

namespace moe {
namespace {

struct LinArgs {
  const int8_t* xq;
  const float* xs;
  const int8_t* wq;
  const float* ws;
  const float* bias;
  bf16_t* out;
  int64_t M, N, K;
};

// One workgroup of WAVES waves per row, kQuantRows of them along the grid's first axis: an
// axis holds fewer than 2^32 threads.
constexpr int64_t kQuantRows = 1 << 20;
template <int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void k_quant_x(const uint4* __restrict__ x, int64_t M, int64_t K,
                                                          uint2* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t red[WAVES];
  const int64_t r = blockIdx.y * kQuantRows + blockIdx.x;
  if (r >= M) return;
  const uint4* src = x + r * (K / 8);
  uint2* dst = codes + r * (K / 8);
  const float s = quant_row_int8<WAVES>(
      K, red, [&](int64_t i, float* f) { unpack8(src[i], f); }, [&](int64_t i, uint2 c) { dst[i] = c; });
  if (threadIdx.x == 0) scales[r] = s;
}

// One workgroup per (16 CT output columns, 16 RT rows): W waves split the
// contraction and their int32 sums meet in LDS.
template <int RT, int CT, int XI, int D, int W>
__global__ __launch_bounds__(W* kWave, 2) void k_linear_rows(LinArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * CT), m0 = (int64_t)blockIdx.y * (RT * 16);
  i32x4_t w[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    // columns past N lie past the buffer; a column tile past N reads the first one
    const int64_t col = n0 + (n0 + 16 * c < a.N ? 16 * c : 0), left = a.N - col;
    w[c] = buffer_of(a.wq + col * a.K, (left < 16 ? left : 16) * a.K);
  }
  const int64_t ml = a.M - m0 < 16 * RT ? a.M - m0 : 16 * RT;
  const i32x4_t x[1] = {buffer_of(a.xq + m0 * a.K, ml * a.K)};
  uint32_t xoff[RT][XI];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < XI; ++j) xoff[r][j] = (16 * r + stream_row(j)) * (uint32_t)a.K;
  i32x4_t acc[CT][RT];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[c][r] = i32x4_t{0, 0, 0, 0};
  const int ns = stream_steps(a.K);
  constexpr int RING = D * kSlot<CT, RT, 1>;
  stream_mfma<true, CT, RT, 1, XI, D>(w, x, xoff, a.K, ns * wave / W, ns * (wave + 1) / W, lds + wave * RING, acc);
  // (the waves' parts take their own rings' place)
  static_assert(RING >= CT * RT * 1024, "parts");
  i32x4_t* red = reinterpret_cast<i32x4_t*>(lds);
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int r = 0; r < RT; ++r) red[wave * (RING / 16) + (c * RT + r) * kWave + lane] = acc[c][r];
  __syncthreads();
  for (int part = wave; part < CT * RT; part += W) {
    const int c = part / RT, r = part % RT;
    i32x4_t s = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < W; ++v) s += red[v * (RING / 16) + part * kWave + lane];
    const int64_t m = m0 + 16 * r + lane % 16, c0 = n0 + 16 * c + 4 * (lane / 16);
    if (m >= a.M) continue;
    const float xs = a.xs[m];
    for (int i = 0; i < 4 && c0 + i < a.N; ++i) {
      float f = (float)s[i] * __fmul_rn(xs, a.ws[c0 + i]);
      if (a.bias) f += a.bias[c0 + i];
      a.out[m * a.N + c0 + i] = (bf16_t)f2bf(f);
    }
  }
}

// The dynamic product of one or two rows in one launch: every workgroup quantises the
// rows for itself, into LDS, behind its first weight loads.  1 x 7168 x 7168 11.3 us
// against 13.4 with a launch for the codes, two rows 12.5 against 13.9; with four rows
// the workgroups' work on the rows costs more than the launch (15.4 against 14.2).
constexpr int kHeldWaves = 8, kHeldPer = 2;
template <int ROWS, int CT, int D>
__global__ __launch_bounds__(kHeldWaves* kWave, 2) void k_linear_held(LinArgs a, const uint4* x) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int W = kHeldWaves, RING = D * kSlot<CT, 0, 0>;
  // dynamic LDS: the rings, the rows' codes, their scales and the quantiser's maxima
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, M = (int)a.M, pitch = held_pitch(a.K);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * CT);
  char* codes = lds + W * RING;
  float* scales = reinterpret_cast<float*>(codes + M * pitch);
  uint32_t* red = reinterpret_cast<uint32_t*>(scales + ROWS);
  i32x4_t w[CT], acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int64_t col = n0 + (n0 + 16 * c < a.N ? 16 * c : 0), left = a.N - col;
    w[c] = buffer_of(a.wq + col * a.K, (left < 16 ? left : 16) * a.K);
    acc[c] = i32x4_t{0, 0, 0, 0};
  }
  const int ns = stream_steps(a.K), row = lane % 16 < M ? lane % 16 : 0;
  stream_held<CT, D>(w, codes + row * pitch + 16 * (lane / 16), a.K, ns * wave / W, ns * (wave + 1) / W,
                              lds + wave * RING, acc, [&] {
    quant_rows_int8<W, ROWS, kHeldPer>(
        M, a.K, red, [&](int r, int64_t i, float* f) { unpack8(x[r * (a.K / 8) + i], f); },
        [&](int r, int64_t i, uint2 c) { *reinterpret_cast<uint2*>(codes + r * pitch + 8 * i) = c; },
        [&](int r, float s) { scales[r] = s; });
    held_pad<W * kWave>(codes, M, a.K, pitch);
    __syncthreads();
  });
  // the waves' parts in their rings' place
  i32x4_t* part = reinterpret_cast<i32x4_t*>(lds);
#pragma unroll
  for (int c = 0; c < CT; ++c) part[wave * (RING / 16) + c * kWave + lane] = acc[c];
  __syncthreads();
  if (wave >= CT || lane % 16 >= M) return;
  i32x4_t s = {0, 0, 0, 0};
#pragma unroll
  for (int v = 0; v < W; ++v) s += part[v * (RING / 16) + wave * kWave + lane];
  const int64_t m = lane % 16, c0 = n0 + 16 * wave + 4 * (lane / 16);
  const float xs = scales[m];
  for (int i = 0; i < 4 && c0 + i < a.N; ++i) {
    float f = (float)s[i] * __fmul_rn(xs, a.ws[c0 + i]);
    if (a.bias) f += a.bias[c0 + i];
    a.out[m * a.N + c0 + i] = (bf16_t)f2bf(f);
  }
}

template <int ROWS, int CT, int D>
moe_status launch_held(const LinArgs& a, const void* x, hipStream_t strm) {
  const int bytes = kHeldWaves * D * kSlot<CT, 0, 0> + (int)a.M * held_pitch(a.K) + ROWS * (1 + kHeldWaves) * 4;
  constexpr auto k = k_linear_held<ROWS, CT, D>;
  if (!lds_allowed<k>(bytes)) return MOE_ERR_HIP;
  hipLaunchKernelGGL(k, dim3((unsigned)((a.N + 16 * CT - 1) / (16 * CT))), dim3(kHeldWaves * kWave), bytes, strm, a,
                     static_cast<const uint4*>(x));
  return launch_status();
}

template <int RT, int CT, int XI, int D, int W>
moe_status launch_rows(const LinArgs& a, hipStream_t strm) {
  constexpr int bytes = W * D * kSlot<CT, RT, 1>;
  static_assert(bytes <= 160 * 1024, "LDS");
  constexpr auto k = k_linear_rows<RT, CT, XI, D, W>;
  if (!lds_allowed<k>(bytes)) return MOE_ERR_HIP;
  hipLaunchKernelGGL(k, dim3((unsigned)((a.N + 16 * CT - 1) / (16 * CT)), (unsigned)((a.M + 16 * RT - 1) / (16 * RT))),
                     dim3(W * kWave), bytes, strm, a);
  return launch_status();
}

typedef int i32x16_t __attribute__((ext_vector_type(16)));

// Tile t of mt x nt tiles: XCD x (workgroups are dealt round-robin) takes the x-th
// eighth of them, in groups of eight row tiles, column by column, so that the tiles in
// flight on an XCD share operands in its L2.
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int BM, int BN, int64_t& m0, int64_t& n0) {
  constexpr int GM = 8;
  const int tiles = mt * nt, x = t & 7, q = tiles >> 3, rem = tiles & 7;
  t = x * q + (x < rem ? x : rem) + (t >> 3);
  const int group = GM * nt, g = t / group, in = t - g * group;
  const int rows = mt - g * GM < GM ? mt - g * GM : GM;
  m0 = (int64_t)(g * GM + in % rows) * BM;
  n0 = (int64_t)(in / rows) * BN;
}

template <int BM, int BN, int WM, int WN, int BK, int S>
__global__ __launch_bounds__(WM* WN* kWave, (BM * BN <= 128 * 128 ? 2 : 1) * WM * WN / 4) void k_linear_tiles(
    LinArgs a, int mt, int nt) {
  constexpr int W = WM * WN, TI = BM / WM / 32, TJ = BN / WN / 32;
  constexpr int RPL = 1024 / BK, CPR = BK / 16;           // rows and chunks of one load
  constexpr int LA = BM / RPL / W, LB = BN / RPL / W;     // loads of a wave and step
  constexpr int kStage = (BM + BN) * BK;
  static_assert(BK == 128, "the swizzle's rows");
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  int64_t m0, n0;
  tile_of(blockIdx.x, mt, nt, BM, BN, m0, n0);
  const uint32_t K = (uint32_t)a.K;
  const int64_t ml = a.M - m0 < BM ? a.M - m0 : BM, nl = a.N - n0 < BN ? a.N - n0 : BN;
  const i32x4_t ra = buffer_of(a.xq + m0 * a.K, ml * a.K), rb = buffer_of(a.wq + n0 * a.K, nl * a.K);
  uint32_t vo[LA + LB], kc[LA + LB];
#pragma unroll
  for (int j = 0; j < LA + LB; ++j) {
    const bool isA = j < LA;
    const int r = ((isA ? wave * LA + j : wave * LB + j - LA)) * RPL + lane / CPR;
    const int64_t lim = (isA ? ml : nl) - 1;
    kc[j] = 16 * swizzle(r, lane % CPR);
    vo[j] = (uint32_t)(r < lim ? r : lim) * K + kc[j];
  }
  const int nk = (int)((a.K + BK - 1) / BK);
  // tiles that share rows start at different steps, so that they do not ask the same
  // L2 channels for the same lines at once
  const int ks = (int)((2 * (m0 / BM + n0 / BN)) % 32) % nk;
  auto issue = [&](int st, int kt) {
    kt = kt + ks < nk ? kt + ks : kt + ks - nk;
    const char* base = lds + st * kStage;
    const uint32_t k0 = (uint32_t)kt * BK;
    if (k0 + BK <= K) {
#pragma unroll
      for (int j = 0; j < LA; ++j) load_lds(ra, base + (wave * LA + j) * 1024, vo[j], k0);
#pragma unroll
      for (int j = 0; j < LB; ++j) load_lds(rb, base + BM * BK + (wave * LB + j) * 1024, vo[LA + j], k0);
    } else {
      // the last, partial step: chunks past the row's end read zeros
#pragma unroll
      for (int j = 0; j < LA; ++j) load_lds(ra, base + (wave * LA + j) * 1024, k0 + kc[j] < K ? vo[j] : kPastBuffer, k0);
#pragma unroll
      for (int j = 0; j < LB; ++j)
        load_lds(rb, base + BM * BK + (wave * LB + j) * 1024, k0 + kc[LA + j] < K ? vo[LA + j] : kPastBuffer, k0);
    }
  };
  i32x16_t acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
  const int wm = wave / WN, wn = wave % WN;
  int ar[TI];
#pragma unroll
  for (int i = 0; i < TI; ++i) ar[i] = wm * (BM / WM) + 32 * i + lane % 32;
  const int br = wn * (BN / WN) + lane % 32;
  // fragments of sub-step kk (32 of K): lane l takes chunk 2 kk + l / 32 of its rows
  i32x4_t fa[2][TI], fb[2][TJ];
  auto read = [&](auto B, const char* stage, int kk) {
    constexpr int b = decltype(B)::value;
    const int c = 2 * kk + lane / 32;
    const char* as = stage + ar[0] * BK + 16 * swizzle(ar[0], c);  // the same for rows 32 apart
    const char* bs = stage + BM * BK + br * BK + 16 * swizzle(br, c);
#pragma unroll
    for (int i = 0; i < TI; ++i) fa[b][i] = *reinterpret_cast<const i32x4_t*>(as + 32 * i * BK);
#pragma unroll
    for (int j = 0; j < TJ; ++j) fb[b][j] = *reinterpret_cast<const i32x4_t*>(bs + 32 * j * BK);
  };
  auto products = [&](auto B) {
    constexpr int b = decltype(B)::value;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[b][j], fa[b][i], acc[i][j], 0, 0, 0);
  };
  constexpr std::integral_constant<int, 0> B0;
  constexpr std::integral_constant<int, 1> B1;
  constexpr int L = LA + LB, KK = BK / 32;
  static_assert(KK % 2 == 0, "fragment buffers alternate");
  // The pipeline: S - 1 steps of loads beyond the current one.  A sub-step's
  // fragments are read while the products of the one before it run; before the last
  // products of a step every wave has its fragments and the next step's tiles have
  // arrived, so one barrier there frees the step's stage for the loads of step
  // kt + S and opens the next one.
#pragma unroll
  for (int p = 0; p < S; ++p)
    if (p < nk) issue(p, p);
  if (S - 1 < nk) __builtin_amdgcn_s_waitcnt(vm_wait(L * (S - 1)));
  else __builtin_amdgcn_s_waitcnt(vm_wait(0));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  int st = 0;
  read(B0, lds, 0);
  for (int kt = 0; kt < nk; ++kt) {
    const char* stage = lds + st * kStage;
#pragma unroll
    for (int kk = 0; kk < KK; kk += 2) {
      read(B1, stage, kk + 1);
      __builtin_amdgcn_sched_barrier(0);
      products(B0);
      __builtin_amdgcn_sched_barrier(0);
      if (kk + 2 < KK) {
        read(B0, stage, kk + 2);
        __builtin_amdgcn_sched_barrier(0);
      }
      else {
        if (kt + S - 1 < nk) __builtin_amdgcn_s_waitcnt(vm_wait(L * (S - 2)));
        else __builtin_amdgcn_s_waitcnt(vm_wait(0));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kt + S < nk) issue(st, kt + S);
        st = st + 1 < S ? st + 1 : 0;
        // (past the last step: stale LDS, not used)
        read(B0, lds + st * kStage, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      products(B1);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __syncthreads();
  // scales and bias, bf16 rows through LDS, whole row pieces out
  constexpr int PITCH = BN * 2 + 16;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int64_t m = m0 + ar[i];
    const float xs = m < a.M ? a.xs[m] : 0.f;
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = wn * (BN / WN) + 32 * j + 8 * q + 4 * (lane / 32);
        float f[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t n = n0 + col + v < a.N ? n0 + col + v : a.N - 1;
          f[v] = (float)acc[i][j][4 * q + v] * __fmul_rn(xs, a.ws[n]);
          if (a.bias) f[v] += a.bias[n];
        }
        *reinterpret_cast<uint2*>(lds + ar[i] * PITCH + col * 2) = make_uint2(pk_bf16(f[0], f[1]), pk_bf16(f[2], f[3]));
      }
  }
  __syncthreads();
  if (a.N % 8 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0) {
    constexpr int VPR = BN / 8;
    for (int v = threadIdx.x; v < BM * VPR; v += W * kWave) {
      const int r = v / VPR, c = v % VPR;
      if (m0 + r < a.M && n0 + c * 8 < a.N)
        *reinterpret_cast<uint4*>(a.out + (m0 + r) * a.N + n0 + c * 8) = *reinterpret_cast<const uint4*>(lds + r * PITCH + c * 16);
    }
  } else {
    for (int v = threadIdx.x; v < BM * BN; v += W * kWave) {
      const int r = v / BN, c = v % BN;
      if (m0 + r < a.M && n0 + c < a.N)
        a.out[(m0 + r) * a.N + n0 + c] = *reinterpret_cast<const bf16_t*>(lds + r * PITCH + c * 2);
    }
  }
}

template <int BM, int BN, int WM, int WN, int BK, int S>
moe_status launch_tiles(const LinArgs& a, hipStream_t strm) {
  const int mt = (int)((a.M + BM - 1) / BM), nt = (int)((a.N + BN - 1) / BN);
  constexpr int stages = S * (BM + BN) * BK, outs = BM * (BN * 2 + 16);
  constexpr int bytes = stages > outs ? stages : outs;
  static_assert(bytes <= 160 * 1024, "LDS");
  constexpr auto k = k_linear_tiles<BM, BN, WM, WN, BK, S>;
  if (!lds_allowed<k>(bytes)) return MOE_ERR_HIP;
  hipLaunchKernelGGL(k, dim3((unsigned)(mt * nt)), dim3(WM * WN * kWave), bytes, strm, a, mt, nt);
  return launch_status();
}

moe_status check_linear(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N <= 0 || K <= 0 || K % 16 != 0) return MOE_ERR_BAD_SHAPE;
  // |sum| <= 127 * 127 * K stays below 2^31 (128 * 128 * K up to K = 131056)
  if (K > 131072) return MOE_ERR_UNSUPPORTED;
  // An axis of a grid holds fewer than 2^32 threads: 512 for each 16 to 64 columns or, on
  // large outputs, each 256 x 256 tile (2^31 for 2^38 outputs, 512 GiB)
  if (M > (int64_t)1 << 24 || N > (int64_t)1 << 24 || M * N > (int64_t)1 << 38) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The operands are read in 16-byte vectors.
bool misaligned(const void* p, const void* q) {
  return (reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) % 16 != 0;
}

// A kernel for codes: its name, as a trace shows it, and its launch.
struct LinKernel {
  const char* name;
  moe_status (*launch)(const LinArgs&, hipStream_t);
};
#define MOE_LIN_KERNEL(kind, ...) \
  LinKernel { "k_linear_" #kind "<" #__VA_ARGS__ ">", launch_##kind<__VA_ARGS__> }

// Up to 48 rows the row kernel, beyond the kernel with the least estimated time (us), from
// what each cost on MI355X with cold weights: a call costs 3 to 3.5, each round of 256
// workgroups (of 64 x 128 tiles too, two of which fit a CU: the fit is by rounds of 256)
// its beginning and end and its part of the contraction, K / 128 steps of the tiled
// kernels, (64 + 16 CT) K bytes of the row kernel at about 95 bytes per ns and CU.
// Measured / estimated: 518 x 2000 x 160 6.2 / 6.4 (64 x 128), 10.2 / 10.1 by rows with CT 2,
// 12.6 / 13.4 with CT 4; 256 x 4096 x 4096 14.1 / 13.2 (rows, CT 4), 16.0 / 16.6 on 64 x 128;
// 512 x 4096 x 7168 25.5 / 24.7 (64 x 128), 56 on 128 x 256; 1024 x 7168 x 7168 66 / 66
// (128 x 256), 99 on 256 x 256; 2000 x 4000 x 512 14.6 / 14 (128 x 256), 15.8 on 64 x 128, 18.8 on
// 256 x 256; 4000 x 8000 x 4096 139 / 140 (256 x 256), 160 on 128 x 256; 4096 x 4096 x 7168
// 114 / 114 (256 x 256), 132 on 128 x 256.
LinKernel linear_kernel(int64_t M, int64_t N, int64_t K) {
  // up to 16 rows: two column tiles for each wave, which halves the rows' share of the
  // loads, where that leaves half a CU's worth of workgroups (16 x 7168 x 7168 12.9
  // against 14.3 us; 1 x 2048 x 7168 8.9 against 6.5 us)
  if (M <= 8 && N < 4096) return MOE_LIN_KERNEL(rows, 1, 1, 1, 2, 8);
  if (M <= 8) return MOE_LIN_KERNEL(rows, 1, 2, 1, 2, 4);
  if (M <= 16 && N < 4096) return MOE_LIN_KERNEL(rows, 1, 1, 2, 2, 8);
  if (M <= 16) return MOE_LIN_KERNEL(rows, 1, 2, 2, 2, 4);
  // more rows: one column tile while those workgroups do not exceed the 256 CUs (20 x 2048
  // x 7168 6.8 against 7.8 us, 37 x 4096 x 4096 6.9 against 7.5; 32 x 7168 x 7168 19 against
  // 14), else two; row tiles as needed (37 x 7168 x 7168 on three 15.3, on four 16.4)
  if (M <= 32 && N <= 4096) return MOE_LIN_KERNEL(rows, 2, 1, 2, 2, 8);
  if (M <= 32) return MOE_LIN_KERNEL(rows, 2, 2, 2, 2, 4);
  if (M <= 48 && N <= 4096) return MOE_LIN_KERNEL(rows, 3, 1, 2, 2, 8);
  if (M <= 48) return MOE_LIN_KERNEL(rows, 3, 2, 2, 1, 8);
  auto up = [](int64_t n, int64_t d) { return (double)((n + d - 1) / d); };
  // (the same with rows past 64, if there are no more row tiles than column tiles: 56 x 2048
  // x 7168 9.3 against 10.9 us, 200 x 1024 x 7168 9.6 against 10.9; 2000 x 128 x 7168 19 against 13)
  if (up(M, 64) * up(N, 16) <= 256 && up(M, 64) <= up(N, 16)) return MOE_LIN_KERNEL(rows, 4, 1, 2, 2, 8);
  const double steps = up(K, 128);
  auto rounds = [&](int bm, int bn) { return up((int64_t)(up(M, bm) * up(N, bn)), 256); };
  const double t[6] = {3 + rounds(64, 32) * (2.2 + K / 980.0),           3 + rounds(64, 64) * (5 + K / 780.0),
                       3.5 + rounds(64, 128) * (2.2 + 0.34 * steps),     3.5 + rounds(128, 128) * (4.5 + 0.6 * steps),
                       3.5 + rounds(128, 256) * (6.5 + steps),           3.5 + rounds(256, 256) * (12 + 1.75 * steps)};
  int best = 0;
  // (the row kernel's workgroups: ceil(M / 64) lie along the grid's second axis)
  for (int i = M > 64 * 65535 ? 2 : 1; i < 6; ++i)
    if (t[i] < t[best] || (best < 2 && M > 64 * 65535)) best = i;
  switch (best) {
    case 0: return MOE_LIN_KERNEL(rows, 4, 2, 2, 1, 8);
    case 1: return MOE_LIN_KERNEL(rows, 4, 4, 2, 2, 4);
    case 2: return MOE_LIN_KERNEL(tiles, 64, 128, 2, 4, 128, 3);
    case 3: return MOE_LIN_KERNEL(tiles, 128, 128, 2, 4, 128, 4);
    case 4: return MOE_LIN_KERNEL(tiles, 128, 256, 2, 4, 128, 3);
    default: return MOE_LIN_KERNEL(tiles, 256, 256, 2, 4, 128, 2);
  }
}

moe_status linear_impl(const LinArgs& a, hipStream_t strm) { return linear_kernel(a.M, a.N, a.K).launch(a, strm); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_linear_int8(int64_t M, int64_t N, int64_t K, const int8_t* xq, const float* xs,
                                      const int8_t* wq, const float* ws, const float* bias, void* out, void* stream) {
  const moe_status st = check_linear(M, N, K);
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  if (!xq || !xs || !wq || !ws || !out) return MOE_ERR_NULL_ARG;
  if (misaligned(xq, wq)) return MOE_ERR_BAD_SHAPE;
  return linear_impl({xq, xs, wq, ws, bias, static_cast<bf16_t*>(out), M, N, K}, as_stream(stream));
}

extern "C" moe_status moe_linear_int8_kernel(int64_t M, int64_t N, int64_t K, const char** name) {
  const moe_status st = check_linear(M, N, K);
  if (st != MOE_OK) return st;
  if (!name) return MOE_ERR_NULL_ARG;
  *name = M == 0 ? "" : linear_kernel(M, N, K).name;
  return MOE_OK;
}

extern "C" moe_status moe_linear_int8_workspace_size(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  const moe_status st = check_linear(M, N, K);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_NULL_ARG;
  // the rows' codes and scales
  *bytes = (size_t)((M * K + 255) / 256 * 256 + (M * 4 + 255) / 256 * 256);
  return MOE_OK;
}

extern "C" moe_status moe_linear_int8_dynamic(int64_t M, int64_t N, int64_t K, const void* x, const int8_t* wq,
                                              const float* ws, const float* bias, void* out, void* workspace,
                                              size_t ws_bytes, void* stream) {
  size_t need = 0;
  const moe_status st = moe_linear_int8_workspace_size(M, N, K, &need);
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  if (!x || !wq || !ws || !out) return MOE_ERR_NULL_ARG;
  if (misaligned(x, wq) || misaligned(workspace, nullptr)) return MOE_ERR_BAD_SHAPE;
  if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
  const LinArgs h = {nullptr, nullptr, wq, ws, bias, static_cast<bf16_t*>(out), M, N, K};
  if (M <= 2 && K <= kHeldPer * 8 * kHeldWaves * kWave) {
    if (M == 2) return launch_held<2, 1, 2>(h, x, as_stream(stream));
    // wide: two column tiles, which halves the workgroups (14336 x 4096 11.8 against 14.0 us)
    return N < 8192 ? launch_held<1, 1, 3>(h, x, as_stream(stream)) : launch_held<1, 2, 2>(h, x, as_stream(stream));
  }
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* xs = reinterpret_cast<float*>(xq + (M * K + 255) / 256 * 256);
  // waves for a row to fit their registers (2048 values each: 4096 rows of 14336, with the
  // product of 1024 columns, 103 us, read twice by four waves 116); eight also where there are
  // few rows (8 rows of 7168: 15.8 against 16.3 us; 8192 of 2048: 44.5 against 39.4)
  auto quant = [&](auto waves) {
    constexpr int W = decltype(waves)::value;
    const dim3 grid((unsigned)std::min(M, kQuantRows), (unsigned)((M + kQuantRows - 1) / kQuantRows));
    hipLaunchKernelGGL((k_quant_x<W>), grid, dim3(W * kWave), 0, as_stream(stream), static_cast<const uint4*>(x), M, K,
                       reinterpret_cast<uint2*>(xq), xs);
    return launch_status();
  };
  const moe_status qs = K > 16384 ? quant(std::integral_constant<int, 16>())
                        : K > 8192 || (K > 4096 && M <= 256) ? quant(std::integral_constant<int, 8>())
                                                             : quant(std::integral_constant<int, 4>());
  if (qs != MOE_OK) return qs;
  return linear_impl({xq, xs, wq, ws, bias, static_cast<bf16_t*>(out), M, N, K}, as_stream(stream));
}
