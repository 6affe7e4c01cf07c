// Queries and keys normalised and rotated to their positions, keys and values into the
// slots of a paged cache (gdn_kv_append).
//
// Bound by the bandwidth of its rows, each read and written once, and for few tokens by
// latency. A warp takes a token, or a part of its heads where there are few tokens: a lane has the
// same 8 columns of a head throughout, so the cosines and sines of its pairs stay in registers,
// and two pieces of 256 columns are on their way while two are worked on, the first before the slot and
// the angles are known. A lane has its pairs' other halves from the lane r / 16 beside it.
// Three CTAs a SM: with four the angles' registers spill. Measured: 16384 tokens of 80 heads of 128, 671 MB, 111 us
// (6.0 TB/s; four pieces that are not ahead of the work 122); 1777 of 32 heads of 256 with norms, 58 MB, 14.7 us,
// 15.0 with rows and slots that are not in L2, a chain of 16 pieces a warp and 110 instructions a piece; 8 tokens 3.1 us.
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

constexpr int kThreads_ = 256, kDeep = 2;

__device__ __forceinline__ unsigned long long turns_of(float f) {
  const double x = fabsf(f), hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
  const double a = x * hi, b = fma(x, hi, -a) + x * lo, r = a - floor(a);
  const unsigned long long u =
      (unsigned long long)(r * 18446744073709551616.0) + (unsigned long long)(long long)(b * 18446744073709551616.0);
  return f < 0.f ? 0ull - u : u;  // 1 - r would lose r's last bits
}

template <int D, bool PAIRS, bool NORM>  // PAIRS: 2 i and 2 i + 1 turn together, else i and i + r / 2
__global__ void __launch_bounds__(kThreads_, 3) kv_append(const AppendParams p) {
  constexpr int kL = D / 8;  // lanes of a head
  __shared__ unsigned long long turn[D / 2];
  const int tid = threadIdx.x, lane = tid & 31, c = lane % kL, half = p.rotary / 2;
  griddep_wait();
  griddep_launch_dependents();
  for (int i = tid; i < half; i += kThreads_) turn[i] = turns_of(p.freq[i]);
  __syncthreads();

  // the lane of the pairs' other halves
  const int shift = half / 8;
  const bool turned = c * 8 < p.rotary, second = c * 8 >= half;
  const int mate = PAIRS || !turned ? lane : second ? lane - shift : lane + shift;
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (NORM && p.qw) wq = *reinterpret_cast<const uint4*>(p.qw + c * 8);
  if (NORM && p.kw) wk = *reinterpret_cast<const uint4*>(p.kw + c * 8);
  const int q_cols = p.Hq * D, k_cols = q_cols + p.Hkv * D, cols = k_cols + p.Hkv * D;
  const int pieces = (cols + 255) / 256, part = (pieces + p.parts - 1) / p.parts;  // of a token; of a warp
  const long long warps = (long long)gridDim.x * (kThreads_ / 32), units = (long long)p.tokens * p.parts;
#pragma unroll 1
  for (long long u = (long long)blockIdx.x * (kThreads_ / 32) + (tid >> 5); u < units; u += warps) {
    const int t = (int)(u / p.parts), first = (int)(u - (long long)t * p.parts) * part, last = min(first + part, pieces);
    const __nv_bfloat16* q = p.q + t * p.ldq;
    const __nv_bfloat16* k = p.k + t * p.ldk - q_cols;
    const __nv_bfloat16* v = p.v + t * p.ldv - k_cols;
    const auto rows_in = [&](int i0, uint4 (&x)[kDeep]) {
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        const int col = (i0 + d) * 256 + lane * 8;
        x[d] = make_uint4(0, 0, 0, 0);
        if (i0 + d < last && col < cols) x[d] = *reinterpret_cast<const uint4*>((col < q_cols ? q : col < k_cols ? k : v) + col);
      }
    };
    uint4 next4[kDeep];
    rows_in(first, next4);
    long long slot = p.slots[t];
    const long long pos = p.pos[t];
    if (slot >= p.num_slots) {
      if (first == 0 && lane == 0 && p.error) atomicCAS(p.error, 0u, (kStatusIndex << 24) | (1u << 16) | (uint32_t)(t & 0xffff));
      slot = -1;
    }
    // a pad row: zero queries, nothing else
    if (slot < 0) {
      for (int col = first * 256 + lane * 8; col < min(last * 256, q_cols); col += 256)
        *reinterpret_cast<uint4*>(p.q_out + t * p.ldqo + col) = make_uint4(0, 0, 0, 0);
      continue;
    }
    float cn[PAIRS ? 4 : 8], sn[PAIRS ? 4 : 8];
    if (turned) {
      const int i0 = PAIRS ? c * 4 : (second ? c * 8 - half : c * 8);
#pragma unroll
      for (int j = 0; j < (PAIRS ? 4 : 8); ++j) {
        const unsigned long long a = (unsigned long long)pos * turn[i0 + j];
        sincospif((float)(int)(a >> 32) * 0x1p-31f, &sn[j], &cn[j]);
        if (!PAIRS && !second) sn[j] = -sn[j];
      }
    }
#pragma unroll 1
    for (int i0 = first; i0 < last; i0 += kDeep) {
      uint4 x4[kDeep];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) x4[d] = next4[d];
      rows_in(i0 + kDeep, next4);
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        if (i0 + d >= last) break;
        const int col = (i0 + d) * 256 + lane * 8;
        const bool is_q = col < q_cols, is_k = !is_q && col < k_cols;
        uint32_t w[4] = {x4[d].x, x4[d].y, x4[d].z, x4[d].w};
        // a piece of values alone, or of heads that neither turn nor are normalised, goes through as it is
        if (__any_sync(0xffffffffu, is_q || is_k) && (NORM || half > 0)) {
          float y[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) y[2 * j] = bf16_lo(w[j]), y[2 * j + 1] = bf16_hi(w[j]);
          if (NORM) {
            const auto squares = [&] {
              float sum = 0.f;
#pragma unroll
              for (int j = 0; j < 8; ++j) sum = fmaf(y[j], y[j], sum);
#pragma unroll
              for (int o = kL / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              return sum * (1.f / D);
            };
            const bool normed = is_q ? p.qw != nullptr : p.kw != nullptr;
            float mean = squares() + p.eps;
            // A head whose squares pass f32's range, or are lost below it, is scaled first. One test for the means from
            // 2^-80 up to 2^120 (1777 tokens of 32 heads of 256 14.7 us; 14.9 with a test for each end and side, 14.4 without).
            constexpr uint32_t kLow = (127 - 80) << 23, kHigh = (127 + 120) << 23;
            if (__any_sync(0xffffffffu, __float_as_uint(mean) - kLow >= kHigh - kLow)) {
              const float by = !normed ? 1.f : !(mean < 0x1p120f) ? 0x1p-100f : mean < 0x1p-80f ? 0x1p80f : 1.f;
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] *= by;
              mean = squares() + p.eps * by * by;
            }
            if (normed) {
              const float scale = rsqrtf(mean);
              const uint32_t n[4] = {is_q ? wq.x : wk.x, is_q ? wq.y : wk.y, is_q ? wq.z : wk.z, is_q ? wq.w : wk.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                y[2 * j] *= scale * (1.f + bf16_lo(n[j]));
                y[2 * j + 1] *= scale * (1.f + bf16_hi(n[j]));
              }
            }
          }
          if (PAIRS) {
            if (turned) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float a = y[2 * j], b = y[2 * j + 1];
                y[2 * j] = a * cn[j] - b * sn[j];
                y[2 * j + 1] = b * cn[j] + a * sn[j];
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float z = __shfl_sync(0xffffffffu, y[j], mate);
              if (turned) y[j] = y[j] * cn[j] + z * sn[j];
            }
          }
          if (is_q || is_k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(y[2 * j], y[2 * j + 1]);
          }
        }
        if (col < cols) {
          __nv_bfloat16* to = is_q ? p.q_out + t * p.ldqo : is_k ? p.k_cache + slot * p.ldkc - q_cols : p.v_cache + slot * p.ldvc - k_cols;
          *reinterpret_cast<uint4*>(to + col) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
}

template <int D, bool PAIRS>
cudaError_t launch(const AppendParams& p, int grid, cudaStream_t s) {
  const Launch l(dim3(grid), kThreads_, 0, true, s);
  return p.qw || p.kw ? cudaLaunchKernelEx(&l.cfg, kv_append<D, PAIRS, true>, p) : cudaLaunchKernelEx(&l.cfg, kv_append<D, PAIRS, false>, p);
}

}  // namespace

cudaError_t launch_kv_append(AppendParams p, int d, bool pairs, cudaStream_t s) {
  // as many warps as run at once; a token's pieces are split where there are fewer tokens
  const long long most = 24LL * sm_count();
  const int pieces = (int)(((long long)(p.Hq + 2 * p.Hkv) * d + 255) / 256);
  p.parts = (int)std::max(1LL, std::min<long long>((pieces + kDeep - 1) / kDeep, most / p.tokens));
  const int grid = (int)((std::min((long long)p.tokens * p.parts, most) + kThreads_ / 32 - 1) / (kThreads_ / 32));
  if (d == 64) return pairs ? launch<64, true>(p, grid, s) : launch<64, false>(p, grid, s);
  if (d == 128) return pairs ? launch<128, true>(p, grid, s) : launch<128, false>(p, grid, s);
  return pairs ? launch<256, true>(p, grid, s) : launch<256, false>(p, grid, s);
}

}  // namespace gdn
