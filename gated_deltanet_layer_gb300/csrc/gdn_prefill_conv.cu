// Causal depthwise conv1d (kernel 4) + SiLU over ragged prompts, with the conv
// state in and out (gdn_prefill_conv).
//
//   out[t][c] = silu(sum_j w[c][j] x[t-3+j][c])
//
// Bound by bandwidth: every input row is read once and every output row written once (4
// bytes a value). A CTA takes one chunk of 64 tokens of one sequence and 1024 channels, 8
// a thread. Its rows come as bulk copies of 2 KB into a ring of 24 in shared memory, four
// CTAs and 192 KB under way on an SM, and a thread walks them with the three older taps in
// registers. 16384 rows of 12288 channels take 132 us, 91% of the measured copy rate (212
// with rows read into registers, 8 in flight: the warps waited for memory 13 cycles of 18).
#include <algorithm>
#include <atomic>

#include "gdn_prefill.cuh"
#include "gdn_tc_pair.cuh"

namespace gdn {
namespace {

constexpr int kConvThreads = 128;
constexpr int kRun = 8;  // rows that arrive together
constexpr int kRowBytes = kConvThreads * 16;
constexpr int kRuns = 3;  // runs of the ring
constexpr int kConvSmem = kRuns * kRun * kRowBytes;

__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
}

// Two values of silu before their rounding to bf16: the fast exponential and reciprocal
// (2^-22) are far below it, and expf with a division took twice the memory's time.
__device__ __forceinline__ uint32_t silu2(float2 y) {
  const float2 t = __fmul2_rn(y, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  const float2 o = __fmul2_rn(y, r);
  return pack_bf16x2(o.x, o.y);
}

__global__ void __launch_bounds__(kConvThreads) conv_kernel(const ConvParams p) {
  extern __shared__ __align__(128) unsigned char rows[];  // [24][2048]
  __shared__ uint64_t full[kRuns];
  griddep_wait();  // for the table of the offsets
  const int place = blockIdx.x;
  int b, e;
  const int s = chunk_seq<true>(p.r, place, &b, &e);
  const int j = place - chunk_first_place(s, b);
  const SeqIn seq = seq_in(p.r, s);
  const bool live = seq_live(p.r, s, seq, b, e, j == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  const int t0 = b + j * kChunk, t1 = min(t0 + kChunk, e);
  const int c0 = blockIdx.y * kConvThreads * 8, c = c0 + threadIdx.x * 8;
  // A place past the sequence's last chunk has no rows, and none before it to
  // take taps from; the first one is always there, for the state.
  if (j > 0 && t0 >= e) return;
  const int n_rows = max(0, t1 - t0);
  const bool mine = c < p.C;
  if (!live) {
    if (mine)
      for (int t = t0; t < t1; ++t)
        *reinterpret_cast<uint4*>(p.out + (long long)t * p.ldo + c) = make_uint4(0, 0, 0, 0);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRuns; ++i) tc::mbar_init(&full[i], 1);
    tc::fence_mbar_init();
  }
  __syncthreads();
  // the first warp's lanes copy the rows of a run into its place of the ring
  const auto fetch = [&](int run) {
    const uint32_t bytes = min(kRowBytes, (p.C - c0) * 2);
    const int first = run * kRun, n = min(kRun, n_rows - first);
    if (n <= 0) return;
    uint64_t* bar = &full[run % kRuns];
    if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(bar, bytes * n);
    __syncwarp();
    if ((int)threadIdx.x < n)
      tc::bulk_load(rows + ((run % kRuns) * kRun + threadIdx.x) * kRowBytes,
                    p.x + (long long)(t0 + first + (int)threadIdx.x) * p.ldx + c0, bytes, bar);
  };
  if (threadIdx.x < 32)
    for (int run = 0; run < kRuns; ++run) fetch(run);
  float2 w[4][4];  // [tap][pair of channels]
  {
    const uint4* wp = reinterpret_cast<const uint4*>(p.w + (size_t)c * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f[4];
      unpack8(mine ? __ldg(wp + i) : make_uint4(0, 0, 0, 0), f);  // two channels' four taps
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k][i] = k & 1 ? make_float2(f[k / 2].y, f[2 + k / 2].y) : make_float2(f[k / 2].x, f[2 + k / 2].x);
    }
  }
  // the three taps before the chunk: rows of the sequence, or the old state
  uint4 h[3] = {};  // packed bf16, oldest first
  const __nv_bfloat16* x = p.x + c;
  if (!mine) {
  } else if (j > 0) {
#pragma unroll
    for (int k = 0; k < 3; ++k) h[k] = __ldg(reinterpret_cast<const uint4*>(x + (long long)(t0 - 3 + k) * p.ldx));
  } else if (seq.in > 0) {
    const uint4* sp = reinterpret_cast<const uint4*>(p.state + ((size_t)seq.in * p.C + c) * 3);
    __align__(16) uint16_t raw[24];
#pragma unroll
    for (int i = 0; i < 3; ++i) reinterpret_cast<uint4*>(raw)[i] = sp[i];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = raw[6 * i + k] | ((uint32_t)raw[6 * i + 3 + k] << 16);
      h[k] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  if (mine && j == 0) {
    // The sequence's new state: its last three inputs. This thread alone reads
    // and writes these channels of the slots, and it has read the old taps, so
    // state_in may be state_out.
    const int n = e - b;
    uint4 l[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int at = n - 3 + k;  // offset in the sequence; before it, the old taps
      l[k] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(x + (long long)(b + at) * p.ldx))
                     : at == -1 ? h[2] : at == -2 ? h[1] : h[0];
    }
    __align__(16) uint16_t raw[24];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t v[4] = {l[k].x, l[k].y, l[k].z, l[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        raw[6 * i + k] = (uint16_t)v[i];
        raw[6 * i + 3 + k] = (uint16_t)(v[i] >> 16);
      }
    }
    uint4* sp = reinterpret_cast<uint4*>(p.state + ((size_t)seq.out * p.C + c) * 3);
#pragma unroll
    for (int i = 0; i < 3; ++i) sp[i] = reinterpret_cast<const uint4*>(raw)[i];
  }
  float2 x0[4], x1[4], x2[4];
  unpack8(h[0], x0);
  unpack8(h[1], x1);
  unpack8(h[2], x2);
  const auto row = [&](int t, const uint4& v) {
    float2 f[4];
    unpack8(v, f);
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[k] = silu2(__ffma2_rn(w[3][k], f[k], __ffma2_rn(w[2][k], x2[k], __ffma2_rn(w[1][k], x1[k], __fmul2_rn(w[0][k], x0[k])))));
      x0[k] = x1[k], x1[k] = x2[k], x2[k] = f[k];
    }
    *reinterpret_cast<uint4*>(p.out + (long long)t * p.ldo + c) = make_uint4(o[0], o[1], o[2], o[3]);
  };
  const unsigned char* at = rows + threadIdx.x * 16;
  bool ok = true;
  for (int run = 0; run * kRun < n_rows; ++run) {
    const int slot = run % kRuns, i = run * kRun, n = min(kRun, n_rows - i);
    ok = tc::mbar_wait(&full[slot], (run / kRuns) & 1) && ok;
    if (mine && ok) {
      if (n == kRun) {
#pragma unroll
        for (int k = 0; k < kRun; ++k) row(t0 + i + k, *reinterpret_cast<const uint4*>(at + (slot * kRun + k) * kRowBytes));
      } else {
        for (int k = 0; k < n; ++k) row(t0 + i + k, *reinterpret_cast<const uint4*>(at + (slot * kRun + k) * kRowBytes));
      }
    }
    if ((run + kRuns) * kRun >= n_rows) continue;
    ok = __syncthreads_and(ok);  // the run is read: its place may be filled again
    if (!ok) {
      // no copy is in flight when the CTA leaves
      for (int r = run; r < run + kRuns; ++r) tc::mbar_wait(&full[r % kRuns], (r / kRuns) & 1);
      break;
    }
    if (threadIdx.x < 32) fetch(run + kRuns);
  }
  if (!ok) record(p.r.error, kStatusDeadline, kWhatWait, s);
}

}  // namespace

cudaError_t launch_conv(const ConvParams& p, cudaStream_t s) {
  static std::atomic<bool> opted[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !opted[dev].load(std::memory_order_relaxed))) {
    e = cudaFuncSetAttribute((const void*)conv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kConvSmem);
    if (e == cudaSuccess && dev < 64) opted[dev].store(true, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(chunk_places(p.r.tokens, p.r.seqs), (p.C / 8 + kConvThreads - 1) / kConvThreads);
  if (p.r.table && (e = launch_offsets(p.r, s)) != cudaSuccess) return e;
  const Launch l(grid, kConvThreads, kConvSmem, p.r.table != nullptr, s);
  return cudaLaunchKernelEx(&l.cfg, conv_kernel, p);
}

}  // namespace gdn
