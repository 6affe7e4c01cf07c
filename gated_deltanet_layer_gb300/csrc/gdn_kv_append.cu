// Queries and keys normalised and rotated to their positions, keys and values into the
// slots of a paged cache (gdn_kv_append).
//
// Bound by the bandwidth of its rows, each read and written once, and for few tokens by
// latency. A CTA takes a few tokens: the cosines and sines of their positions go through
// shared memory once for all heads; then every head's row is D / 8 lanes of 16 bytes, four rows
// of a lane on their way at a time, and a lane has its pair's other half from the lane
// r / 16 beside it.
//
// Angles. pos f is wanted modulo a turn, to f32's accuracy at any position. f / (2 pi) is
// a 64-bit binary fraction of a turn (in two double terms, so right to its last bits), and
// its product with the position, cut to 64 bits, is the fraction again: whole turns
// fall off by themselves.
#include <algorithm>

#include "gdn_attn.cuh"
#include "gdn_host.h"
#include "gdn_prefill.cuh"

namespace gdn {
namespace {

constexpr int kThreads_ = 256, kDeep = 4;
constexpr int kMaxTokens = 4;  // of a CTA

__device__ __forceinline__ unsigned long long turns_of(float f) {
  const double x = f, hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
  const double a = x * hi, b = fma(x, hi, -a) + x * lo, r = a - floor(a);
  return (unsigned long long)(r * 18446744073709551616.0) + (unsigned long long)(long long)(b * 18446744073709551616.0);
}

template <int D, bool PAIRS>  // PAIRS: 2 i and 2 i + 1 turn together, else i and i + r / 2
__global__ void __launch_bounds__(kThreads_) kv_append(const AppendParams p) {
  constexpr int kL = D / 8, kGroups = kThreads_ / kL;
  __shared__ unsigned long long turn[D / 2];
  __shared__ float2 cs[kMaxTokens][D / 2];
  const int tid = threadIdx.x, half = p.rotary / 2;
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = blockIdx.x * p.per, count = min(p.per, p.tokens - t0);
  for (int i = tid; i < half; i += kThreads_) turn[i] = turns_of(p.freq[i]);
  __syncthreads();
  for (int x = tid; x < count * half; x += kThreads_) {
    const int t = x / half, i = x - t * half;
    const unsigned long long a = (unsigned long long)(long long)p.pos[t0 + t] * turn[i];
    float sn, cn;
    sincospif((float)(int)(a >> 32) * 0x1p-31f, &sn, &cn);
    cs[t][i] = make_float2(cn, sn);
  }
  __syncthreads();

  const int lane = tid & 31, c = tid % kL, heads = p.Hq + 2 * p.Hkv, items = count * heads;
  // the lane of the pairs' other halves, and the sign of the sine there
  const int shift = half / 8;
  const bool turned = c * 8 < p.rotary, second = c * 8 >= half;
  const int mate = PAIRS || !turned ? lane : second ? lane - shift : lane + shift;
  const int mate_c = PAIRS || !turned ? c : second ? c - shift : c + shift;
  float wq[8], wk[8];
  const auto weights = [&](const __nv_bfloat16* w, float (&o)[8], int at) {
    const uint4 v = w ? *reinterpret_cast<const uint4*>(w + at * 8) : make_uint4(0, 0, 0, 0);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) o[2 * j] = 1.f + bf16_lo(u[j]), o[2 * j + 1] = 1.f + bf16_hi(u[j]);
  };
  weights(p.qw, wq, c);
  weights(p.kw, wk, c);
  float mq[8], mk[8];
  weights(p.qw, mq, mate_c);
  weights(p.kw, mk, mate_c);

#pragma unroll 1
  for (int base = 0; base < items; base += kGroups * kDeep) {
    uint4 v[kDeep];
    int tok[kDeep], head[kDeep];
    long long slot[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int item = base + k * kGroups + tid / kL;
      tok[k] = item < items ? item / heads : -1;
      v[k] = make_uint4(0, 0, 0, 0);
      if (tok[k] >= 0) {
        head[k] = item - tok[k] * heads;
        const long long t = t0 + tok[k];
        slot[k] = p.slots[t];
        if (slot[k] >= p.num_slots) {
          if (head[k] == 0 && c == 0 && p.error) atomicCAS(p.error, 0u, (kStatusIndex << 24) | (1u << 16) | (uint32_t)(t & 0xffff));
          slot[k] = -1;
        }
        const __nv_bfloat16* row = head[k] < p.Hq           ? p.q + t * p.ldq + head[k] * D
                                   : head[k] < p.Hq + p.Hkv ? p.k + t * p.ldk + (head[k] - p.Hq) * D
                                                            : p.v + t * p.ldv + (head[k] - p.Hq - p.Hkv) * D;
        if (slot[k] >= 0) v[k] = *reinterpret_cast<const uint4*>(row + c * 8);
      }
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const bool on = tok[k] >= 0, is_q = on && head[k] < p.Hq, is_k = on && !is_q && head[k] < p.Hq + p.Hkv;
      uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w}, w[4];
      float x[8], scale = 1.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[2 * j] = bf16_lo(u[j]), x[2 * j + 1] = bf16_hi(u[j]);
      const bool norm = is_q ? p.qw != nullptr : is_k && p.kw != nullptr;
      if (p.qw || p.kw) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
        for (int o = kL / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (norm) scale = 1.f / sqrtf(sum * (1.f / D) + p.eps);
      }
      if (!PAIRS) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __shfl_sync(0xffffffffu, u[j], mate);
      }
      if (!on) continue;
      if (is_q || is_k) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = norm ? x[j] * scale * (is_q ? wq[j] : wk[j]) : x[j];
        if (turned) {
          const float2* a = cs[tok[k]];
          if (PAIRS) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = a[c * 4 + j];
              const float e = y[2 * j], o = y[2 * j + 1];
              y[2 * j] = e * f.x - o * f.y;
              y[2 * j + 1] = o * f.x + e * f.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 f = a[(second ? mate_c : c) * 8 + j];
              const float raw = j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
              const float z = norm ? raw * scale * (is_q ? mq[j] : mk[j]) : raw;
              y[j] = second ? y[j] * f.x + z * f.y : y[j] * f.x - z * f.y;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = pack_bf16x2(y[2 * j], y[2 * j + 1]);
      }
      const uint4 r = make_uint4(u[0], u[1], u[2], u[3]);
      if (is_q)
        *reinterpret_cast<uint4*>(p.q_out + (long long)(t0 + tok[k]) * p.ldqo + head[k] * D + c * 8) =
            slot[k] >= 0 ? r : make_uint4(0, 0, 0, 0);
      else if (slot[k] >= 0)
        *reinterpret_cast<uint4*>(is_k ? p.k_cache + slot[k] * p.ldkc + (head[k] - p.Hq) * D + c * 8
                                       : p.v_cache + slot[k] * p.ldvc + (head[k] - p.Hq - p.Hkv) * D + c * 8) = r;
    }
  }
}

template <int D>
cudaError_t launch(const AppendParams& p, bool pairs, int grid, cudaStream_t s) {
  const Launch l(dim3(grid), kThreads_, 0, true, s);
  return pairs ? cudaLaunchKernelEx(&l.cfg, kv_append<D, true>, p) : cudaLaunchKernelEx(&l.cfg, kv_append<D, false>, p);
}

}  // namespace

cudaError_t launch_kv_append(AppendParams p, int d, bool pairs, cudaStream_t s) {
  p.per = std::max(1, std::min(kMaxTokens, p.tokens / (2 * sm_count())));
  const int grid = (p.tokens + p.per - 1) / p.per;
  return d == 64 ? launch<64>(p, pairs, grid, s) : d == 128 ? launch<128>(p, pairs, grid, s) : launch<256>(p, pairs, grid, s);
}

}  // namespace gdn
