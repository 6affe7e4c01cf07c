// act(x W^T + bias) + residual with W in 4 bits (gdn_linear_w4): a few rows of x, bound by
// the bandwidth of the weights and the instructions that unpack them.
//
// y[m][n] = sum over groups of scale[n][g] sum_k value[n][k] x[m][k], value = code - zero or E2M1.
// Products by mma.sync (16 weight rows x 8 rows of x x 16 columns) in bf16 with f32 sums, a
// group at a time, then scale times the group's sum in f32: a value has at most 8 bits, so
// no weight is rounded, and x is taken as it is.
//
// The order of the columns within a group of 32 is free as long as x has the same: a
// lane's eight codes are one 32-bit word, its eight of x the 16 bytes beside them. Whole numbers: the
// codes' bytes as bf16 are c 2^-133, one multiply-add makes (c - zero) 2^-6 of two. E2M1: the two
// bytes of a bf16 from tables of eight, by permutes whose selectors are the codes themselves.
//
// A CTA's warps are R x S: R groups of 16 weight rows, as many as give every SM one CTA, and S shares of
// the columns, as many as there are warps left, whose sums are added up in shared memory at the end.
// A warp's codes come through a ring of its own (cp.async), its scales and zeros four groups at
// a time through registers, and x to the lanes as it is, from L1. Through shared memory, pieces of all
// shares at a time, its room was what bounded S: 16 rows of 1024 x 8192 33 us, 6.4 now; 8 rows of
// 8192 x 8192 20.8 and 14.7.
//
// 8, 16 or 32 rows of x at a time, the weights once for each: as many as there are, fewer at a time where the groups are too few
// for the SMs all the same (up to two a SM): 33 rows of 1037 x 1056 8.2 us with 32 at a time, 5.6 with 16. 64 at a
// time leave too few registers: 64 rows of 8192 x 8192 77 us, 58 with two passes.
//
// Measured with the weights from memory, as a server has them (and with the same weights over and over, part of them in L2):
// 8 rows of 20480 x 8192 whole numbers 31.4 us (25.0), 2.8 TB/s; MXFP4 37.4 (35.1); 16 of 5120 x 5120 14.0 (10.7); 64 of
// 8192 x 8192 91 (58.6); 2560 x 8192, one row, MXFP4 10.4 (9.8), whole numbers 9.7 (8.4). Figures above are the latter. A SM's
// warps issue an instruction every other cycle, 45 for 512 weights (unpack 22,
// the scales 8, loads and addresses 8), and 160 groups of rows are two for a CTA, which leaves 72 SMs idle.
#include <algorithm>
#include <type_traits>

#include "gdn_host.h"
#include "gdn_prefill.cuh"
#include "gdn_tc_ptx.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kStep = 256;              // columns of a stage
constexpr int kStages = 4;
constexpr int kPitch = kStep / 2;       // bytes of a stage's row; its 16-byte pieces permuted, against bank conflicts
constexpr int kStageBytes = 16 * kPitch, kRing = kStages * kStageBytes;  // of a warp

// Warps of a CTA: what the registers allow.
template <int MT>
constexpr int warps() { return MT <= 2 ? 20 : 16; }

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// (v & mask) | w.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(w));
  return r;
}
// Eight whole numbers (c - zero) 2^-6 as bf16; less: -zero 2^-6 twice.
__device__ __forceinline__ void unpack_int(uint32_t w, uint32_t less, uint32_t (&o)[4]) {
  const uint32_t ev = w & 0x0f0f0f0fu, od = (w >> 4) & 0x0f0f0f0fu;  // codes 0 2 4 6, 1 3 5 7
  // a byte and its sign, which is 0, of each: bf16 subnormals
  o[0] = fma_bf16x2(prmt(ev, od, 0xC480), 0x7f007f00u, less);
  o[1] = fma_bf16x2(prmt(ev, od, 0xD591), 0x7f007f00u, less);
  o[2] = fma_bf16x2(prmt(ev, od, 0xE6A2), 0x7f007f00u, less);
  o[3] = fma_bf16x2(prmt(ev, od, 0xF7B3), 0x7f007f00u, less);
}
// Eight E2M1 values as bf16.
__device__ __forceinline__ void unpack_e2m1(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t up = w << 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // 0, 1/2, 1, 3/2, 2, 3, 4, 6: 0000 3F00 3F80 3FC0 4000 4040 4080 40C0
    const uint32_t sel = (h ? w >> 16 : w) & 0x7777u;
    const uint32_t lo = prmt(0xC0800000u, 0xC0804000u, sel), hi = prmt(0x3F3F3F00u, 0x40404040u, sel);
    // bit 7 of these bytes: the codes' signs
    const uint32_t top = and_or(prmt(up, w, h ? 0x7362 : 0x5140), 0x80808080u, hi);
    o[2 * h] = prmt(lo, top, 0x5140);
    o[2 * h + 1] = prmt(lo, top, 0x7362);
  }
}
// 2^(e - 127), NaN for 255, as f32.
__device__ __forceinline__ uint32_t e8m0(uint32_t e) { return max(e << 23, 0x00400000u) | (e == 255 ? 0x00400000u : 0u); }
__device__ __forceinline__ float act_f(float y, int act) {
  if (act == 0) return y;
  const float s = act == 1 ? y : y * fmaf(0.07135481627f, y * y, 1.595769122f);
  return __fdividef(y, 1.0f + __expf(-s));
}

// FMT 0: whole numbers with zeros, 1: E2M1. GPS: scale groups of a stage (8, 4, 2). MT: 8 rows of x.
template <int FMT, int GPS, int MT>
__global__ void __launch_bounds__(32 * warps<MT>(), 1) linear_w4(const W4Params p) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int kNT = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int R = p.row_groups, S = p.shares, rg = warp % R, sl = warp / R;
  unsigned char* const ring = smem + warp * kRing;
  const int m0 = blockIdx.y * MT * 8, M = min(MT * 8, p.M - m0);
  const int all = (p.K + kStep - 1) / kStep;
  const int each = (all + S - 1) / S;  // stages of a share
  const int s0 = min(sl * each, all), s1 = min(s0 + each, all);
  const int n0 = (blockIdx.x * R + rg) * 16;
  const long long row0 = min(n0 + g, p.N - 1), row1 = min(n0 + g + 8, p.N - 1);
  const int groups = p.K / p.group;  // of a row
  griddep_wait();
  griddep_launch_dependents();

  // the lane's four 16-byte pieces of a stage's codes, of every fourth row
  const unsigned char* from[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    from[i] = p.codes + (long long)min(n0 + (lane >> 3) + 4 * i, p.N - 1) * (p.K / 2) + (long long)s0 * (kStep / 2) + (lane & 7) * 16;
  const uint32_t to = smem_u32(ring + (lane >> 3) * kPitch);
  const auto codes_in = [&](int st) {
    if (st < s1) {
      const bool on = st * kStep + (lane & 7) * 32 < p.K;
      const uint32_t at = to + (st & (kStages - 1)) * kStageBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         at + i * (4 * kPitch) + (((lane & 7) ^ ((lane >> 3) + 4 * i & 7)) << 4)),
                     "l"(on ? from[i] : p.codes), "r"(on ? 16 : 0)
                     : "memory");
        from[i] += kStep / 2;
      }
    }
    cp_async_commit();
  };
  // Scales (and zeros) of four groups of the two rows: a lane's t-th.
  const auto scale_in = [&](int quad, uint32_t (&v)[2]) {
    const int at = quad * 4 + t;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[e] = 0;
      if (at < groups) {
        const long long i = (e ? row1 : row0) * groups + at;
        if (FMT == 1)
          v[e] = __ldg(static_cast<const uint8_t*>(p.scales) + i);
        else
          v[e] = (uint32_t)__ldg(static_cast<const unsigned short*>(p.scales) + i) << 16 | (p.zeros ? __ldg(p.zeros + i) : 8u);
      }
    }
  };
  constexpr int kQuad = GPS < 4 ? 4 / GPS : 1, kQuads = GPS > 4 ? GPS / 4 : 1;  // stages of four groups; fours of a stage
  constexpr int kAhead = 2 * kQuads;  // fours that are on their way
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) codes_in(s0 + i);
  uint32_t sc[kAhead][2];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) scale_in(s0 / kQuad * kQuads + i, sc[i]);

  float acc[MT][4] = {};
  // full: all its columns are there
  const auto stage = [&](int st, auto full) {
    codes_in(st + kStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const unsigned char* codes = ring + (st & (kStages - 1)) * kStageBytes + g * kPitch + t * 4;
    const int k0 = st * kStep + t * 8;  // the lane's first column
    const int in_quad = kQuad > 1 ? (st % kQuad) * GPS : 0;  // the stage's first scale group, of the lanes' four
    float z[MT][4], f[2];
    uint32_t less[2];
#pragma unroll
    for (int q = 0; q < kStep / 32; ++q) {
      constexpr int PER = kStep / 32 / GPS;  // groups of 32 of a scale group
      if (q % PER == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t v = __shfl_sync(0xffffffffu, FMT == 1 ? e8m0(sc[q / PER / 4][e]) : sc[q / PER / 4][e], (lane & 28) + in_quad + q / PER % 4);
          if (FMT == 1) {
            f[e] = __uint_as_float(v);
          } else {
            f[e] = __uint_as_float(v & 0xffff0000u);
            const float u = (float)(v & 0xffff) * -0x1p-6f;
            less[e] = pack_bf16x2(u, u);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) z[mt][0] = z[mt][1] = z[mt][2] = z[mt][3] = 0.f;
      }
      uint4 y[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (!full) y[mt] = make_uint4(0, 0, 0, 0);
        if (full || (mt * 8 < M && k0 + q * 32 < p.K))
          y[mt] = __ldg(reinterpret_cast<const uint4*>(p.x + (long long)(m0 + min(mt * 8 + g, M - 1)) * p.ldx + k0 + q * 32));
      }
      const int at = (q ^ g) << 4;
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(codes + at);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(codes + 8 * kPitch + at);
      uint32_t v0[4], v1[4];
      if (FMT == 1) {
        unpack_e2m1(w0, v0);
        unpack_e2m1(w1, v1);
      } else {
        unpack_int(w0, less[0], v0);
        unpack_int(w1, less[1], v1);
      }
      const uint32_t a[4] = {v0[0], v1[0], v0[1], v1[1]}, b[4] = {v0[2], v1[2], v0[3], v1[3]};
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt > 0 && mt * 8 >= M) break;  // no such rows
        mma_bf16_16816(z[mt], a, y[mt].x, y[mt].y);
        mma_bf16_16816(z[mt], b, y[mt].z, y[mt].w);
      }
      if (q % PER == PER - 1) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[mt][0] = fmaf(f[0], z[mt][0], acc[mt][0]);
          acc[mt][1] = fmaf(f[0], z[mt][1], acc[mt][1]);
          acc[mt][2] = fmaf(f[1], z[mt][2], acc[mt][2]);
          acc[mt][3] = fmaf(f[1], z[mt][3], acc[mt][3]);
        }
      }
    }
    if ((st + 1) % kQuad == 0) {
#pragma unroll
      for (int i = 0; i < kAhead - kQuads; ++i) sc[i][0] = sc[i + kQuads][0], sc[i][1] = sc[i + kQuads][1];
#pragma unroll
      for (int i = kAhead - kQuads; i < kAhead; ++i) scale_in((st + 1) / kQuad * kQuads + i, sc[i]);
    }
    __syncwarp();
  };
  // With 32 rows a test before each load pays: without one they are all asked for at once, and the registers that
  // they come to are missing elsewhere (64 rows of 8192 x 8192 58 us, 86 without). With fewer it costs 5 to 8%.
  const int whole = MT <= 2 ? min(s1, p.K / kStep) : s0;
  int st = s0;
  if (MT <= 2)
#pragma unroll 1
    for (; st < whole; ++st) stage(st, std::true_type());
#pragma unroll 1
  for (; st < s1; ++st) stage(st, std::false_type());
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // the shares' sums, over the rings: [share][row of x][weight row]
  const int W = R * 16;
  float* out = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = mt * 8 + 2 * t + (i & 1);
      if (m < M) out[(sl * M + m) * W + rg * 16 + g + 8 * (i >> 1)] = FMT == 1 ? acc[mt][i] : acc[mt][i] * 64.f;
    }
  }
  __syncthreads();
  for (int i = tid; i < M * W; i += kNT) {
    const int m = i / W, n = i - m * W, col = blockIdx.x * W + n;
    if (col >= p.N) continue;
    float y = 0.f;
    for (int sh = 0; sh < S; ++sh) y += out[(sh * M + m) * W + n];
    if (p.bias) y += bf16_to_f(p.bias[col]);
    y = act_f(y, p.act);
    const long long row = m0 + m;
    if (p.residual) y += bf16_to_f(p.residual[row * p.ldr + col]);
    p.out[row * p.ldo + col] = __float2bfloat16_rn(y);
  }
}

template <int FMT, int GPS, int MT>
cudaError_t launch(W4Params p, cudaStream_t s) {
  constexpr int kMost = warps<MT>();
  static_assert(kMost * kRing <= 232448, "227 KB of shared memory a CTA");
  static_assert(16 * MT * 8 * 4 <= kRing, "the shares' sums");
  const cudaError_t e = opt_in<linear_w4<FMT, GPS, MT>>(kMost * kRing);
  if (e != cudaSuccess) return e;
  const int passes = (p.M + MT * 8 - 1) / (MT * 8), rows16 = (p.N + 15) / 16, steps = (p.K + kStep - 1) / kStep;
  const int R = (int)std::min<long long>(kMost, ((long long)rows16 * passes + sm_count() - 1) / sm_count());
  const int S = std::max(1, std::min(kMost / R, steps));
  p.row_groups = R;
  p.shares = S;
  const Launch l(dim3((rows16 + R - 1) / R, passes), 32 * R * S, R * S * kRing, true, s);
  return cudaLaunchKernelEx(&l.cfg, linear_w4<FMT, GPS, MT>, p);
}
template <int FMT, int GPS>
cudaError_t by_rows(const W4Params& p, cudaStream_t s) {
  // passes of fewer rows where there are SMs for them
  const auto fits = [&](int rows) { return (p.N + 15LL) / 16 * ((p.M + rows - 1) / rows) <= 2 * sm_count(); };
  if (p.M <= 8 || fits(8)) return launch<FMT, GPS, 1>(p, s);
  return p.M <= 16 || fits(16) ? launch<FMT, GPS, 2>(p, s) : launch<FMT, GPS, 4>(p, s);
}

}  // namespace

cudaError_t launch_linear_w4(const W4Params& p, cudaStream_t s) {
  if (p.mx) return by_rows<1, 8>(p, s);
  return p.group == 32 ? by_rows<0, 8>(p, s) : p.group == 64 ? by_rows<0, 4>(p, s) : by_rows<0, 2>(p, s);
}

}  // namespace gdn
