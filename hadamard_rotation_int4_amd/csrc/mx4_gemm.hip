// Product of two MXFP4 operands, C = A W^T, on the matrix cores' scaled fp4
// instructions.
//
// What is computed: C[m][n] = sum over blocks j of 2^(Ea[m][j] + Ew[n][j]) times
// the sum of the 32 products of the block's codes, in fp32, rounded once to
// the output type.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds row l % 16 of its operand and
// the 32 codes (16 bytes) of block l / 16 of the step's four, with that block's
// scale byte.  The weights are the first operand, so that a lane's four results
// are four consecutive columns of one row of C.
#include "mx4_device.h"

namespace hr {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;      // format code of the instruction's operands

__device__ __forceinline__ v8i fp4_operand(const uint4& x) {
  return (v8i){(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
}

// One element of C, rounded to its type.
__device__ __forceinline__ void store_c(const Mx4GemmArgs& p, int64_t at, float v) {
  if (p.dtype == kDtF32) reinterpret_cast<float*>(p.c)[at] = v;
  else if (p.dtype == kDtBf16) reinterpret_cast<__bf16*>(p.c)[at] = (__bf16)v;
  else reinterpret_cast<_Float16*>(p.c)[at] = (_Float16)v;
}

// 16 columns and 16 MT rows of C a workgroup; its waves take the steps of 128
// along K in turn and their sums are joined in LDS, in the waves' order.
constexpr int kRowWaves = 8;

template <int MT>
__global__ __launch_bounds__(64 * kRowWaves) void mx4_gemm_rows_kernel(Mx4GemmArgs p) {
  __shared__ v4f part[kRowWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, kb = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int blocks = p.K / kMxBlock, steps = (blocks + 3) / 4;
  const int64_t wrow = n0 + r < p.N ? n0 + r : p.N - 1;     // rows past the end: the last again, stored nowhere
  int64_t arow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) arow[t] = m0 + 16 * t + r < p.M ? m0 + 16 * t + r : p.M - 1;
  v4f acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = wave; s < steps; s += kRowWaves) {
    const int j = 4 * s + kb;
    const bool live = j < blocks;                           // past the end: zero codes and scales
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const uint4 wc = live ? *reinterpret_cast<const uint4*>(p.w + wrow * (p.K / 2) + 16 * j) : z;
    const int ws = live ? p.sw[wrow * blocks + j] : 0;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint4 ac = live ? *reinterpret_cast<const uint4*>(p.a + arow[t] * (p.K / 2) + 16 * j) : z;
      const int as = live ? p.sa[arow[t] * blocks + j] : 0;
      acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(wc), fp4_operand(ac), acc[t], kFp4, kFp4, 0, ws,
                                                                0, as);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 64; i += 64 * kRowWaves) {
    const int t = i >> 6, l = i & 63;
    v4f c = part[0][t][l];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) c += part[w][t][l];
    const int64_t m = m0 + 16 * t + (l & 15), n = n0 + 4 * (l >> 4);
    if (m >= p.M) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (n + v < p.N) store_c(p, m * p.N + n + v, c[v]);
  }
}

hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, hipStream_t s) {
  const unsigned cols = (unsigned)((a.N + 15) / 16);
  if (a.M <= 16)
    hipLaunchKernelGGL((mx4_gemm_rows_kernel<1>), dim3(cols, (unsigned)((a.M + 15) / 16)), dim3(64 * kRowWaves), 0, s, a);
  else
    hipLaunchKernelGGL((mx4_gemm_rows_kernel<4>), dim3(cols, (unsigned)((a.M + 63) / 64)), dim3(64 * kRowWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace hr
