// act(x W^T + bias) + residual with W in 4 bits (gdn_linear_w4): a few rows of x, bound by
// the bandwidth of the weights.
//
// y[m][n] = sum over groups of scale[n][g] (sum_k code[n][k] x[m][k] - zero[n][g] sum_k x[m][k]).
// Products by mma.sync (16 weight rows x 8 rows of x x 16 columns) in f16 with f32 sums, a
// group at a time, then scale times the group's sum in f32, so no weight is ever rounded.
//
// x as f16: every row times a power of two that takes its largest value to 2^14 .. 2^15, which
// keeps bf16's 8 bits down to 2^-27 of that value.
// Codes as f16. 4-bit whole numbers: 0x6400 | code is 1024 + code, and with the code four bits
// further up 1024 + 16 code, so eight codes are four ANDs with an OR and one shift. The
// columns of the second kind take x / 16, and what the 1024s add is known from sums of x: a group's
// sum starts from minus that and minus zero times sum x. E2M1: a conversion of the hardware's, exact.
// The order of the columns within a group of 32 is free as long as x has the same: a
// lane's eight codes are one 32-bit word, and x is laid out in shared memory as the lanes want it.
//
// A CTA takes 128 weight rows, 16 a warp, and a share of the columns; the CTAs of a cluster
// share the columns and add their sums through distributed shared memory, in order.
#include <cuda_fp16.h>

#include <algorithm>

#include "gdn_host.h"
#include "gdn_prefill.cuh"
#include "gdn_tc_pair.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kW = 8, kNT = kW * 32;
constexpr int kRowsN = 16 * kW;     // weight rows of a CTA
constexpr int kStep = 128;          // columns of a stage
constexpr int kStages = 8;
constexpr int kPitch = kStep / 2 + 16;  // bytes of a stage's row: its codes, and 16 against bank conflicts

// Columns of x in shared memory at a time.
template <int MT>
constexpr int chunk() { return MT <= 2 ? 1024 : MT == 4 ? 512 : 256; }

template <int MT>
struct W4Smem {
  unsigned char ring[kW][kStages][16 * kPitch];
  uint4 x[chunk<MT>() / 32][MT][32];               // [group of 32][8 rows][lane]: 8 columns of a row as f16
  float4 sums[chunk<MT>() / 32][MT][4];            // [group][8 rows][t]: what to start from, of rows 2 t and 2 t + 1: 1024s' part, sum x
  float out[MT * 8][kRowsN];
  float factor[MT * 8], unfactor[MT * 8];
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (v & mask) | 0x6400 in both halves.
__device__ __forceinline__ uint32_t and_or_1024(uint32_t v, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(0x64006400u));
  return r;
}
// Two E2M1 codes of a byte as f16.
__device__ __forceinline__ uint32_t e2m1x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 b, x, y, z;\n\tmov.b32 {b, x, y, z}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(byte));
  return r;
}
// Scales take 2^-15 with them, so that with x at up to 2^16 no sum is larger than what it stands
// for; bf16's 8 bits and powers of two are exact at any size of theirs.
constexpr float kDown = 0x1p-15f;
__device__ __forceinline__ float e8m0(uint32_t e) {  // 2^(e - 127) of them
  return __uint_as_float(e < 16 ? 0x80u << e : e == 255 ? 0x7fc00000u : (e - 15) << 23);
}
__device__ __forceinline__ float act_f(float y, int act) {
  if (act == 0) return y;
  const float s = act == 1 ? y : y * fmaf(0.07135481627f, y * y, 1.595769122f);
  return __fdividef(y, 1.0f + __expf(-s));
}

// FMT 0: whole numbers with zeros, 1: E2M1. GPS: scale groups of a stage (4, 2, 1).
template <int FMT, int GPS, int MT>
__global__ void __launch_bounds__(kNT) linear_w4(const W4Params p) {
  extern __shared__ unsigned char raw[];
  W4Smem<MT>& s = *reinterpret_cast<W4Smem<MT>*>(raw);
  constexpr int KC = chunk<MT>();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const int m0 = blockIdx.y * MT * 8, M = min(MT * 8, p.M - m0);
  const int all = (p.K + kStep - 1) / kStep;
  const int s0 = (int)((long long)all * rank / p.split), s1 = (int)((long long)all * (rank + 1) / p.split);
  const int n0 = tile * kRowsN + warp * 16;
  const long long row0 = min(n0 + g, p.N - 1), row1 = min(n0 + g + 8, p.N - 1);
  const int groups = p.K / p.group;  // of a row
  griddep_wait();
  griddep_launch_dependents();

  const auto issue = [&](int st) {
    if (st < s1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane + 32 * i) >> 2, q = lane & 3, k = st * kStep + q * 32;
        const unsigned char* src = p.codes + (long long)min(n0 + r, p.N - 1) * (p.K / 2) + k / 2;
        const bool on = k < p.K;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         smem_u32(s.ring[warp][(st - s0) % kStages] + r * kPitch + q * 16)),
                     "l"(on ? src : p.codes), "r"(on ? 16 : 0)
                     : "memory");
      }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) issue(s0 + i);

  // the rows' powers of two
  for (int m = warp; m < MT * 8; m += kW) {
    uint32_t top = 0;
    if (m < M) {
      const __nv_bfloat16* x = p.x + (long long)(m0 + m) * p.ldx;
      for (int k = s0 * kStep + lane * 8; k < min(s1 * kStep, p.K); k += 256) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + k);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a = (u[j] >> 7) & 0xff, b = (u[j] >> 23) & 0xff;
          if (a < 255) top = max(top, a);
          if (b < 255) top = max(top, b);
        }
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) {
      const int e = top == 0 ? 0 : max(-112, min(127, 141 - (int)top));
      s.factor[m] = __uint_as_float((uint32_t)(e + 127) << 23);
      s.unfactor[m] = __uint_as_float((uint32_t)(15 - e + 127) << 23);
    }
  }
  float acc[MT][4] = {};
  __syncthreads();

  int st = s0;
#pragma unroll 1
  for (int c0 = s0; c0 < s1; c0 += KC / kStep) {
    const int c1 = min(c0 + KC / kStep, s1);
    // x of the chunk
    for (int i = tid; i < (c1 - c0) * 4 * MT * 32; i += kNT) {
      const int l = i & 31, mt = (i >> 5) % MT, gr = (i >> 5) / MT, m = mt * 8 + (l >> 2), k = c0 * kStep + gr * 32 + (l & 3) * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (m < M && k < p.K) v = *reinterpret_cast<const uint4*>(p.x + (long long)(m0 + m) * p.ldx + k);
      const float f = s.factor[m];
      const float y[8] = {bf16_lo(v.x) * f, bf16_hi(v.x) * f, bf16_lo(v.y) * f, bf16_hi(v.y) * f,
                          bf16_lo(v.z) * f, bf16_hi(v.z) * f, bf16_lo(v.w) * f, bf16_hi(v.w) * f};
      const auto h2 = [](float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
      };
      if (FMT == 1) {
        s.x[gr][mt][l] = make_uint4(h2(y[0], y[1]), h2(y[2], y[3]), h2(y[4], y[5]), h2(y[6], y[7]));
      } else {
        constexpr float q = 0.0625f;
        const uint4 o = make_uint4(h2(y[0], y[4]), h2(y[1] * q, y[5] * q), h2(y[2], y[6]), h2(y[3] * q, y[7] * q));
        s.x[gr][mt][l] = o;
        // the sums of what is multiplied: of the first kind's columns, and of the second's
        const auto sum = [](uint32_t a, uint32_t b) {
          const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a)), w = __half22float2(*reinterpret_cast<const __half2*>(&b));
          return (u.x + u.y) + (w.x + w.y);
        };
        float one = sum(o.x, o.z), two = sum(o.y, o.w);
        float start = (one + two) * 1024.f, x = one + 16.f * two;
        start += __shfl_xor_sync(0xffffffffu, start, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        start += __shfl_xor_sync(0xffffffffu, start, 2);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if ((l & 3) == 0) reinterpret_cast<float2*>(&s.sums[gr][mt][0])[l >> 2] = make_float2(start, x);
      }
    }
    __syncthreads();
#pragma unroll 1
    for (; st < c1; ++st) {
      issue(st + kStages - 1);
      float sc[GPS][2], zr[GPS][2];
#pragma unroll
      for (int q = 0; q < GPS; ++q) {
        const int at = st * GPS + q;
        const bool on = at < groups;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const long long i = (e ? row1 : row0) * groups + (on ? at : 0);
          if (FMT == 1) {
            sc[q][e] = on ? e8m0(static_cast<const uint8_t*>(p.scales)[i]) : 0.f;
          } else {
            sc[q][e] = on ? bf16_to_f(static_cast<const __nv_bfloat16*>(p.scales)[i]) * kDown : 0.f;
            zr[q][e] = p.zeros ? (float)p.zeros[i] : 8.f;
          }
        }
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const unsigned char* codes = s.ring[warp][(st - s0) % kStages];
      float c[MT][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        constexpr int PER = 4 / GPS;  // groups of 32 of a scale group
        const int gr = (st - c0) * 4 + q, sg = q / PER;
        if (q % PER == 0) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (FMT == 1) {
              c[mt][0] = c[mt][1] = c[mt][2] = c[mt][3] = 0.f;
            } else {
              float4 z = s.sums[gr][mt][t];
#pragma unroll
              for (int i = 1; i < PER; ++i) {
                const float4 y = s.sums[gr + i][mt][t];
                z.x += y.x, z.y += y.y, z.z += y.z, z.w += y.w;
              }
              c[mt][0] = -fmaf(zr[sg][0], z.y, z.x);
              c[mt][1] = -fmaf(zr[sg][0], z.w, z.z);
              c[mt][2] = -fmaf(zr[sg][1], z.y, z.x);
              c[mt][3] = -fmaf(zr[sg][1], z.w, z.z);
            }
          }
        }
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(codes + g * kPitch + q * 16 + t * 4);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(codes + (g + 8) * kPitch + q * 16 + t * 4);
        uint32_t a[4], b[4];
        if (FMT == 1) {
          a[0] = e2m1x2(w0), a[1] = e2m1x2(w1), a[2] = e2m1x2(w0 >> 8), a[3] = e2m1x2(w1 >> 8);
          b[0] = e2m1x2(w0 >> 16), b[1] = e2m1x2(w1 >> 16), b[2] = e2m1x2(w0 >> 24), b[3] = e2m1x2(w1 >> 24);
        } else {
          const uint32_t lo = 0x000f000fu, hi = 0x00f000f0u, v0 = w0 >> 8, v1 = w1 >> 8;
          a[0] = and_or_1024(w0, lo), a[1] = and_or_1024(w1, lo), a[2] = and_or_1024(w0, hi), a[3] = and_or_1024(w1, hi);
          b[0] = and_or_1024(v0, lo), b[1] = and_or_1024(v1, lo), b[2] = and_or_1024(v0, hi), b[3] = and_or_1024(v1, hi);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 x = s.x[gr][mt][lane];
          mma_f16(c[mt], a, x.x, x.y);
          mma_f16(c[mt], b, x.z, x.w);
        }
        if (q % PER == PER - 1) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            acc[mt][0] = fmaf(sc[sg][0], c[mt][0], acc[mt][0]);
            acc[mt][1] = fmaf(sc[sg][0], c[mt][1], acc[mt][1]);
            acc[mt][2] = fmaf(sc[sg][1], c[mt][2], acc[mt][2]);
            acc[mt][3] = fmaf(sc[sg][1], c[mt][3], acc[mt][3]);
          }
        }
      }
      __syncwarp();
    }
    __syncthreads();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m = mt * 8 + 2 * t, n = warp * 16 + g;
    s.out[m][n] = acc[mt][0] * s.unfactor[m];
    s.out[m + 1][n] = acc[mt][1] * s.unfactor[m + 1];
    s.out[m][n + 8] = acc[mt][2] * s.unfactor[m];
    s.out[m + 1][n + 8] = acc[mt][3] * s.unfactor[m + 1];
  }
  if (p.split > 1)
    cluster_sync();
  else
    __syncthreads();
  // this CTA's share of the columns, over all of the cluster's sums
  const int per = (kRowsN + p.split - 1) / p.split, b = rank * per, e = min(b + per, kRowsN);
  for (int i = tid; i < M * per; i += kNT) {
    const int m = i / per, n = b + i % per, col = tile * kRowsN + n;
    if (n >= e || col >= p.N) continue;
    float y = 0.f;
    if (p.split > 1) {
#pragma unroll 1
      for (int r = 0; r < p.split; ++r) y += ld_cluster_f(map_rank(&s.out[m][n], r));
    } else {
      y = s.out[m][n];
    }
    if (p.bias) y += bf16_to_f(p.bias[col]);
    y = act_f(y, p.act);
    const long long row = m0 + m;
    if (p.residual) y += bf16_to_f(p.residual[row * p.ldr + col]);
    p.out[row * p.ldo + col] = __float2bfloat16_rn(y);
  }
  if (p.split > 1) cluster_sync();  // no CTA leaves while its part is read
}

template <int FMT, int GPS, int MT>
cudaError_t launch(W4Params p, cudaStream_t s) {
  const size_t smem = sizeof(W4Smem<MT>);
  static_assert(sizeof(W4Smem<MT>) <= 232448, "227 KB of shared memory a CTA");
  const cudaError_t e = opt_in<linear_w4<FMT, GPS, MT>>(smem);
  if (e != cudaSuccess) return e;
  const int tiles = (p.N + kRowsN - 1) / kRowsN, passes = (p.M + MT * 8 - 1) / (MT * 8), steps = (p.K + kStep - 1) / kStep;
  p.split = std::max(1, std::min({8, 2 * sm_count() / (tiles * passes), steps}));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.split * tiles, passes);
  cfg.blockDim = dim3(kNT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = p.split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_w4<FMT, GPS, MT>, p);
}
template <int FMT, int GPS>
cudaError_t by_rows(const W4Params& p, cudaStream_t s) {
  return p.M <= 8 ? launch<FMT, GPS, 1>(p, s) : p.M <= 16 ? launch<FMT, GPS, 2>(p, s) : p.M <= 32 ? launch<FMT, GPS, 4>(p, s)
                                                                                                : launch<FMT, GPS, 8>(p, s);
}

}  // namespace

cudaError_t launch_linear_w4(const W4Params& p, cudaStream_t s) {
  if (p.mx) return by_rows<1, 4>(p, s);
  return p.group == 32 ? by_rows<0, 4>(p, s) : p.group == 64 ? by_rows<0, 2>(p, s) : by_rows<0, 1>(p, s);
}

}  // namespace gdn
