// The matrix product on 8-bit integers with a scale for each token and each
// output channel, moe_linear_int8: out[m, n] = bf16((sum_k xq[m, k] wq[n, k]) *
// (xs[m] * ws[n]) + bias[n]), the sum exact in int32; and its dynamic form, which
// first quantises bf16 rows by the rule of moe_quant_rows_int8.
//
// k_linear_rows: one workgroup per (16 output columns, up to 64 rows).  Its waves
// split the contraction, each streaming its part of the 16 weight rows from
// memory into the matrix cores (stream_mfma.hpp); the int32 partial sums meet in
// LDS, where their order does not matter.  Bound: HBM, N * K bytes of weights.
#include "stream_mfma.hpp"

namespace moe {
namespace {

constexpr int kRowWaves = 8;

struct LinArgs {
  const int8_t* xq;
  const float* xs;
  const int8_t* wq;
  const float* ws;
  const float* bias;
  bf16_t* out;
  int64_t M, N, K;
};

// one workgroup per row
__global__ __launch_bounds__(256) void k_quant_x(const uint4* __restrict__ x, int64_t K, uint2* __restrict__ codes,
                                                 float* __restrict__ scales) {
  __shared__ float red[4];
  const int64_t r = blockIdx.x;
  const uint4* src = x + r * (K / 8);
  uint2* dst = codes + r * (K / 8);
  const float s = quant_row_int8<4>(
      K, red, [&](int64_t i, float* f) { unpack8(src[i], f); }, [&](int64_t i, uint2 c) { dst[i] = c; });
  if (threadIdx.x == 0) scales[r] = s;
}

template <int RT>
__global__ __launch_bounds__(kRowWaves* kWave) void k_linear_rows(LinArgs a) {
  __shared__ i32x4_t red[kRowWaves][RT][kWave];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (RT * 16);
  // a column or row past the end reads the last one
  const uint32_t K = (uint32_t)a.K, nl = (uint32_t)(a.N - 1 - n0), ml = (uint32_t)(a.M - 1 - m0);
  const char* w[1] = {reinterpret_cast<const char*>(a.wq) + n0 * a.K};
  const char* x[1] = {reinterpret_cast<const char*>(a.xq) + m0 * a.K};
  const uint32_t row = lane % 16, chunk = 16 * (lane / 16);
  const uint32_t woff[1] = {(row < nl ? row : nl) * K + chunk};
  uint32_t xoff[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const uint32_t m = 16 * r + row;
    xoff[r] = (m < ml ? m : ml) * K + chunk;
  }
  i32x4_t acc[1][RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[0][r] = i32x4_t{0, 0, 0, 0};
  const int ns = stream_steps(a.K);
  stream_mfma<true, 1, RT, 1, RT == 1 ? 8 : (RT == 2 ? 4 : 2)>(w, woff, x, xoff, a.K, ns * wave / kRowWaves,
                                                              ns * (wave + 1) / kRowWaves, acc);
#pragma unroll
  for (int r = 0; r < RT; ++r) red[wave][r][lane] = acc[0][r];
  __syncthreads();
  if (wave >= RT) return;
  i32x4_t s = {0, 0, 0, 0};
#pragma unroll
  for (int v = 0; v < kRowWaves; ++v) s += red[v][wave][lane];
  const int64_t m = m0 + 16 * wave + lane % 16, c0 = n0 + 4 * (lane / 16);
  if (m >= a.M) return;
  const float xs = a.xs[m];
  for (int i = 0; i < 4 && c0 + i < a.N; ++i) {
    float f = (float)s[i] * __fmul_rn(xs, a.ws[c0 + i]);
    if (a.bias) f += a.bias[c0 + i];
    a.out[m * a.N + c0 + i] = (bf16_t)f2bf(f);
  }
}

moe_status check_linear(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N <= 0 || K <= 0 || K % 16 != 0) return MOE_ERR_BAD_SHAPE;
  // |sum| <= 127 * 127 * K stays below 2^31
  if (K > 131072) return MOE_ERR_UNSUPPORTED;
  if (M > (int64_t)1 << 24 || N > (int64_t)1 << 24) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The operands are read in 16-byte vectors.
bool misaligned(const void* p, const void* q) {
  return (reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) % 16 != 0;
}

moe_status linear_impl(const LinArgs& a, hipStream_t strm) {
  const unsigned nt = (unsigned)((a.N + 15) / 16);
  const int rt = a.M <= 16 ? 1 : (a.M <= 32 ? 2 : 4);
  const dim3 grid(nt, (unsigned)((a.M + rt * 16 - 1) / (rt * 16))), block(kRowWaves * kWave);
  if (rt == 1) hipLaunchKernelGGL(k_linear_rows<1>, grid, block, 0, strm, a);
  else if (rt == 2) hipLaunchKernelGGL(k_linear_rows<2>, grid, block, 0, strm, a);
  else hipLaunchKernelGGL(k_linear_rows<4>, grid, block, 0, strm, a);
  return launch_status();
}

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
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* xs = reinterpret_cast<float*>(xq + (M * K + 255) / 256 * 256);
  hipLaunchKernelGGL(k_quant_x, dim3((unsigned)M), dim3(256), 0, as_stream(stream), static_cast<const uint4*>(x), K,
                     reinterpret_cast<uint2*>(xq), xs);
  return linear_impl({xq, xs, wq, ws, bias, static_cast<bf16_t*>(out), M, N, K}, as_stream(stream));
}
