// The gated delta rule over ragged prompts (gdn_prefill_delta): the recurrent
// form, one token after the other, for sequences of up to kRecurrentMax tokens;
// it also writes the rows of padding.
//
// One CTA for each (sequence, value head). A warp keeps 32 rows of the state
// S[dv][dk] in registers, a lane the columns lane*E .. lane*E + E - 1 of all of
// them (E = dk / 32), so a row of the pool is one coalesced load. Per token:
// S <- e^g S and the partial dots S k; a transposing butterfly (31 shuffles)
// leaves row i's sum in lane i, which forms u_i = beta (v_i - (S k)_i); u is
// broadcast back, S += u k^T, and o = S q the same way. All f32.
// One token is bound by the state's read and write: 129 requests of 64 heads in f32 take
// 174 us, 93% of the measured copy rate. A further token takes 0.9 us a CTA, two
// transposing sums and the broadcasts being a third of its instructions.
#include <algorithm>

#include "gdn_prefill.cuh"

namespace gdn {
namespace {

template <int E>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, float (&f)[E]) {
  if constexpr (E == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  } else {
    const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(p));
    f[0] = bf16_lo(v), f[1] = bf16_hi(v);
  }
}

template <int E, bool BF16>
__device__ __forceinline__ void load_state(const void* base, size_t at, float (&f)[E]) {
  if constexpr (BF16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + at;
    if constexpr (E == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    } else {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
      f[0] = bf16_lo(v), f[1] = bf16_hi(v);
    }
  } else {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (E == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p);
      f[0] = v.x, f[1] = v.y;
    }
  }
}

template <int E, bool BF16>
__device__ __forceinline__ void store_state(void* base, size_t at, const float (&f)[E]) {
  if constexpr (BF16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + at;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    else
      *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(f[0], f[1]);
  } else {
    float* p = static_cast<float*>(base) + at;
    if constexpr (E == 4)
      *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else
      *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  }
}

// Lane i receives the sum over the lanes of their v[i].
__device__ __forceinline__ float transpose_sum(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const bool upper = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = upper ? v[i] : v[i + w];
      const float keep = upper ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
    }
  }
  return v[0];
}

template <int D, bool BF16>
__global__ void __launch_bounds__(D) recurrent_kernel(const DeltaParams p) {
  constexpr int E = D / 32, W = D / 32;
  __shared__ float red[2][W];
  griddep_wait();               // for the table of the offsets, which the chunked form's first kernel reads as well
  griddep_launch_dependents();  // that kernel touches nothing of this one's
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.x, h = blockIdx.y;
  const SeqIn seq = seq_in(p.r, s);
  int b, e;
  seq_rows(p.r, s, seq, &b, &e);
  const bool live = seq_live(p.r, s, seq, b, e, h == 0 && threadIdx.x == 0);
  if (h == 0 && threadIdx.x == 0 && s < p.r.seqs && p.plan)
    p.plan[s] = make_int4(b, live && e - b > kRecurrentMax ? e : b, seq.in, seq.out);
  if (live && e - b > kRecurrentMax) return;  // the chunked form's
  const int row = threadIdx.x;  // the dv row this lane finishes
  if (p.order && s == p.r.seqs && h == 0) {
    // the sequences' order for the chunked form, longest first (bad offsets: any order)
    __shared__ unsigned len[kSorted];
    for (int i = row; i < s; i += D) len[i] = (unsigned)__ldg(p.r.cu + i + 1) - (unsigned)__ldg(p.r.cu + i);
    __syncthreads();
    for (int i = row; i < s; i += D) {
      int rank = 0;
      for (int j = 0; j < s; ++j) rank += len[j] > len[i] || (len[j] == len[i] && j < i);
      p.order[rank] = i;
    }
  }
  if (!live) {
    // padding: zero rows, 16 bytes a thread
    for (int t = b + threadIdx.x / (D / 8); t < e; t += 8)
      *reinterpret_cast<uint4*>(p.out + (long long)t * p.ldo + h * D + threadIdx.x % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int kh = h / p.group;
  float S[32][E] = {};
  if (seq.in > 0) {
    const size_t at = (((size_t)seq.in * p.Hv + h) * D + warp * 32) * D + lane * E;
#pragma unroll
    for (int i = 0; i < 32; ++i) load_state<E, BF16>(p.state, at + (size_t)i * D, S[i]);
  }
  const float rate = expf(p.A_log[h]), shift = bf16_to_f(p.dt_bias[h]);
  const float gw = p.z ? bf16_to_f(p.gnorm_w[row]) : 0.f;
  for (int t = b; t < e; ++t) {
    const __nv_bfloat16* x = p.qkv + (long long)t * p.ldqkv;
    float q[E], k[E], v = bf16_to_f(x[2 * p.Hk * D + h * D + row]);
    load_bf16<E>(x + kh * D + lane * E, q);
    load_bf16<E>(x + (p.Hk + kh) * D + lane * E, k);
    const __nv_bfloat16* ba = p.ba + (long long)t * p.ldba;
    const float beta = sigmoid_f(bf16_to_f(ba[h]));
    const float decay = expf(-rate * softplus_f(bf16_to_f(ba[p.Hv + h]) + shift));
    float qq = 0.f, kk = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) qq = fmaf(q[i], q[i], qq), kk = fmaf(k[i], k[i], kk);
    qq = warp_sum(qq), kk = warp_sum(kk);
    const float rq = p.q_scale / sqrtf(qq + p.l2_eps), rk = 1.0f / sqrtf(kk + p.l2_eps);
#pragma unroll
    for (int i = 0; i < E; ++i) q[i] *= rq, k[i] *= rk;
    float d[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      d[i] = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) {
        S[i][c] *= decay;
        d[i] = fmaf(S[i][c], k[c], d[i]);
      }
    }
    const float u = beta * (v - transpose_sum(d));
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float ui = __shfl_sync(0xffffffffu, u, i);
      d[i] = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) {
        S[i][c] = fmaf(ui, k[c], S[i][c]);
        d[i] = fmaf(S[i][c], q[c], d[i]);
      }
    }
    float o = transpose_sum(d);
    if (p.z) {
      const float part = warp_sum(o * o);
      if (lane == 0) red[t & 1][warp] = part;
      __syncthreads();  // two buffers: one barrier a token is enough
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) sum += red[t & 1][i];
      const float z = bf16_to_f(p.z[(long long)t * p.ldz + h * D + row]);
      o = o / sqrtf(sum * (1.0f / D) + p.gnorm_eps) * gw * silu_f(z);
    }
    p.out[(long long)t * p.ldo + h * D + row] = __float2bfloat16_rn(o);
  }
  const size_t at = (((size_t)seq.out * p.Hv + h) * D + warp * 32) * D + lane * E;
#pragma unroll
  for (int i = 0; i < 32; ++i) store_state<E, BF16>(p.state, at + (size_t)i * D, S[i]);
}

template <int D>
cudaError_t launch_d(const DeltaParams& p, bool state_bf16, cudaStream_t s) {
  const dim3 grid(p.r.seqs + 1, p.Hv);  // the last sequence is the pad rows
  if (p.r.table) {
    const cudaError_t e = launch_offsets(p.r, s);
    if (e != cudaSuccess) return e;
  }
  const Launch l(grid, D, 0, p.r.table != nullptr, s);
  return cudaLaunchKernelEx(&l.cfg, state_bf16 ? recurrent_kernel<D, true> : recurrent_kernel<D, false>, p);
}

}  // namespace

cudaError_t launch_delta(const DeltaParams& whole, int d, bool state_bf16, unsigned char* ws, cudaStream_t s) {
  DeltaParams p = whole;
  const bool chunks = p.r.seqs > 0 && std::min(p.r.max_len, p.r.tokens) > kRecurrentMax;
  if (!chunks) p.order = nullptr, p.plan = nullptr;
  const cudaError_t e = d == 128 ? launch_d<128>(p, state_bf16, s) : launch_d<64>(p, state_bf16, s);
  if (e != cudaSuccess || !chunks) return e;
  return launch_delta_chunks(p, d, state_bf16, ws, s);
}

}  // namespace gdn
