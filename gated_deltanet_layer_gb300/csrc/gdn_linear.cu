// act(x W^T + bias) + residual (gdn_linear).
#include "gdn_prefill.cuh"

namespace gdn {
namespace {

constexpr int kT = 64, kK = 32;

__device__ __forceinline__ float act_f(float y, int act) {
  if (act == 1) return silu_f(y);
  if (act == 2) return 0.5f * y * (1.0f + tanhf(0.7978845608028654f * (y + 0.044715f * y * y * y)));
  return y;
}

// 64 x 64 outputs a CTA, 4 x 4 a thread, f32 FMA from shared tiles.
__global__ void __launch_bounds__(256) linear_kernel(const LinearParams p) {
  __shared__ float xs[kK][kT + 1], ws[kK][kT + 1];
  const int m0 = blockIdx.y * kT, n0 = blockIdx.x * kT;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kK) {
    for (int i = threadIdx.x; i < kT * kK; i += 256) {
      const int r = i / kK, k = i % kK;
      const bool in = k0 + k < p.K;
      xs[k][r] = in && m0 + r < p.M ? bf16_to_f(p.x[(long long)(m0 + r) * p.ldx + k0 + k]) : 0.f;
      ws[k][r] = in && n0 + r < p.N ? bf16_to_f(p.w[(long long)(n0 + r) * p.ldw + k0 + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[k][ty * 4 + i], ws[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      float y = act_f(acc[i][j] + (p.bias ? bf16_to_f(p.bias[n]) : 0.f), p.act);
      if (p.residual) y += bf16_to_f(p.residual[(long long)m * p.ldr + n]);
      p.out[(long long)m * p.ldo + n] = __float2bfloat16_rn(y);
    }
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, cudaStream_t s) {
  const dim3 grid((p.N + kT - 1) / kT, (p.M + kT - 1) / kT);
  linear_kernel<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
