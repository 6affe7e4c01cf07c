// The gated delta rule over ragged prompts (gdn_prefill_delta): the chunked
// form on the tensor cores, for sequences of more than kRecurrentMax tokens.
//
// A chunk is 64 tokens. With G_i the running sum of the log gates in the chunk,
// S0 the state before it and k, q normalised,
//   u_i = beta_i (v_i - e^(G_i) S0 k_i - sum_{j<i} e^(G_i-G_j) (k_i.k_j) u_j),
// so with L_ij = beta_i e^(G_i-G_j) (k_i.k_j) for j < i and T = (I + L)^-1
//   R = diag(beta) (V - diag(e^G) K S0^T),   U = T R,
//   O = diag(e^G) Q S0^T + tril(e^(G_i-G_j) q_i.k_j) U,
//   S = e^(G_C) S0 + sum_j e^(G_C-G_j) u_j k_j^T.
//
// Two kernels. prepare_kernel does what does not depend on the state, for every
// chunk at once: norms, gates, K K^T and Q K^T, T. delta_kernel walks a sequence's
// chunks, one CTA for each (sequence, value head), with S^T as a [dv][dk] f32
// accumulator in TMEM.
//
// Precision. The state and all sums are f32. What multiplies the state runs as f16
// products of two-term splits, x = hi + lo (22 bits), accumulated in f32: S hi+lo by
// k; T hi+lo by R hi+lo (without lo lo); U hi+lo by k. Raw q and k are bf16, so as f16,
// after a power of two for each token, they are exact down to 2^-17 of the token's
// largest value. The output's own terms (S by q, the causal products by U) take two
// each as well: a q across the keys, or repeated keys, make large values cancel there.
// f16's range: every row of S^T (a TMEM lane, one thread) has a power of two for the
// state and one for U, from bounds that hold throughout the chunk. With |k| <= 1 and
// beta <= 1 a token's step S <- e^g S (I - beta k k^T) + beta v k^T does not lengthen a
// row by more than beta |v|, so over a chunk
//   |S'| <= e^(G_C) |S0| + sum_j e^(G_C-G_j) beta_j |v_j|  (every e^(G_C-G_j) u_j too),
//   |u_j|, |R_j| <= max(beta) (max |v| + |S0| + sum beta |v|);
// |T| <= 1 takes the constant 2^12. Two terms reach 2^-39 of such a bound.
//
// Values that are not finite stay where the definition has them: a row of S^T knows
// the first token whose v, k or gates are not, multiplies zeros from there on, and
// stores NaN from that token on instead, so no earlier token sees 0 x NaN.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "gdn_prefill.cuh"
#include "gdn_tc_pair.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr float kScaleT = 4096.f;   // of T's f16 images
constexpr int kImg = 4 * 8192;      // T hi, T lo, causal products hi, lo: 64 x 64 f16 each
enum { S_BETA, S_C1, S_CU, S_W, S_CQG, S_CQ, S_END, S_COUNT };  // arrays of 64 floats beside them
constexpr int kHeadBytes = kImg + S_COUNT * 256;
// S_END: [0] e^(G_C), [1] (an int) the first token whose k or gates are not finite,
// else 64, [2] the largest beta

template <int D>
constexpr int kq_bytes() { return 2 * kChunk * D * 2; }

struct ChunkParams {
  DeltaParams p;
  unsigned char* kq;    // [place][Hk] f16 images of k and q
  unsigned char* head;  // [place][Hv] images and scalars
};

// Byte of (row, column) in a K-major operand image of 64 f16 columns, 128-byte swizzle.
__device__ __forceinline__ int swz(int row, int col) { return row * 128 + ((((col >> 3) ^ row) & 7) << 4) + (col & 7) * 2; }

__device__ __forceinline__ uint32_t pack_h2(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// y = hi + lo, two f16 each
__device__ __forceinline__ void split2(float2 y, uint32_t* hi, uint32_t* lo) {
  const __half2 h = __float22half2_rn(y);
  *hi = pack_h2(h);
  *lo = pack_h2(__float22half2_rn(__ffma2_rn(__half22float2(h), make_float2(-1.f, -1.f), y)));
}

// D[tmem] (+)= A[smem or tmem] B[smem], f16 operands, f32 accumulation.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// kind::f16 with f16 inputs (formats 0) and an f32 accumulator; mn_b: B's rows
// are K and its columns N.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool mn_b) {
  return (1u << 4) | ((mn_b ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Descriptor of an N-major operand in the 128-byte swizzled layout: K rows of 128
// bytes (64 N values), 8-row groups 1024 bytes apart, the next 64 N values `next`
// bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t next) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(next >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const float (&v)[32]) {
  uint32_t r[16];
#pragma unroll
  for (int h = 0; h < 32; h += 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[h + i]);
    tmem_st16(t + h, r);
  }
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Power of two f with |x| f < 2^14 for every |x| <= b, kept where f, 1 / f and the
// ratios of two of them are ordinary floats.
__device__ __forceinline__ float row_scale(float b) {
  const int e = min(max((int)(__float_as_uint(b) >> 23) & 0xff, 64), 254);
  return __uint_as_float((uint32_t)(267 - e) << 23);
}
__device__ __forceinline__ float inverse_pow2(float f) { return __uint_as_float((254u << 23) - __float_as_uint(f)); }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// A sum kept as hi + lo (two f32), so differences of sums of large gates keep their
// small bits.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float e = (a.hi - (s - t)) + (b.hi - t) + a.lo + b.lo;
  const float h = s + e;
  return Two{h, e - (h - s)};
}

// ------------------------------------------------------------------ prepare

constexpr int kPrepThreads = 256;
constexpr int kLStride = 68;  // floats of a row of L: 16-byte rows, apart in banks
constexpr int kXStride = 36;

template <int D>
struct alignas(1024) PrepSmem {
  union {
    unsigned char kq[D / 64][128 * 128];  // rows k 0..63, q 0..63, in atoms of 64 columns
    unsigned char t[2][2][8192];          // then T of two heads, hi and lo
    float x[2][32 * kXStride];            // and between, a product on T's way
  };
  unsigned char a[2][2][8192];  // causal products of two heads, hi and lo
  float m[2][64 * kLStride];    // L, then T in its place
  float scal[2][S_COUNT][64];
  float ghi[2][64], glo[2][64];  // running sums of the log2 gates
  float bj[2][64];               // 2^(G of the 16-block's end - G_j) / norm of k_j
  float top[2][64];              // of a row of the causal products, by column halves
  float rn[128];                 // 1 / norm of the f16 rows (k, q)
  int bad[64];                   // k not finite
  uint64_t done;
  uint32_t tmem;
};

// x[i] += sum_l A[i][l] B[l][c..c+3] for R rows i of A, l0 <= l < l1 (multiples of 4).
template <int R>
__device__ __forceinline__ void mac4(float4 (&x)[R], const float* A, int lda, const float* B, int ldb, int l0, int l1) {
#pragma unroll 1
  for (int l = l0; l < l1; l += 4) {
    float4 a[R];
#pragma unroll
    for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(A + i * lda + l);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(B + (l + k) * ldb);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float w = k == 0 ? a[i].x : k == 1 ? a[i].y : k == 2 ? a[i].z : a[i].w;
        x[i].x = fmaf(w, v.x, x[i].x), x[i].y = fmaf(w, v.y, x[i].y);
        x[i].z = fmaf(w, v.z, x[i].z), x[i].w = fmaf(w, v.w, x[i].w);
      }
    }
  }
}
__device__ __forceinline__ float4 minus(float4 v) { return make_float4(-v.x, -v.y, -v.z, -v.w); }

template <int D>
__global__ void __launch_bounds__(kPrepThreads, 2) prepare_kernel(const ChunkParams c) {
  const DeltaParams& p = c.p;
  extern __shared__ unsigned char raw[];
  PrepSmem<D>& s = *reinterpret_cast<PrepSmem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int place = blockIdx.x, kh = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sq = chunk_seq(p.r, place);
  int b, e, in, out;
  seq_rows(p.r, sq, &b, &e);
  const int t0 = b + (place - chunk_first_place(p.r, sq)) * kChunk, n = min(kChunk, e - t0);
  if (n <= 0 || e - b <= kRecurrentMax || !seq_slots(p.r, sq, false, &in, &out)) return;
  if (warp == 0) tmem_alloc(&s.tmem, 64);
  if (tid == 0) {
    mbar_init(&s.done, 1);
    fence_mbar_init();
  }
  // k and q rows: norms, and f16 images scaled by a power of two each
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
#pragma unroll 4
  for (int i = 0; i < 16; i += kRows) {
    const int row = warp * 16 + i + lane / kLanes, tok = row & 63, col = (lane % kLanes) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (tok < n)
      v = __ldg(reinterpret_cast<const uint4*>(p.qkv + (long long)(t0 + tok) * p.ldqkv + (row < 64 ? p.Hk + kh : kh) * D + col));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8], ss = 0.f, mx = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = bf16_lo(w[j]), f[2 * j + 1] = bf16_hi(w[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss), mx = fmaxf(mx, fabsf(f[j]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    // 2^ex > mx >= 2^(ex-1)
    const int ex = min(max((int)(__float_as_uint(mx) >> 23) - 126, -126), 127);
    const float up = __uint_as_float((uint32_t)(127 + ex) << 23), down = __uint_as_float((uint32_t)(127 - ex) << 23);
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = pack_h2(__floats2half2_rn(f[2 * j] * down, f[2 * j + 1] * down));
    *reinterpret_cast<uint4*>(s.kq[col >> 6] + swz(row, col & 63)) = make_uint4(h[0], h[1], h[2], h[3]);
    if (lane % kLanes == 0) {
      s.rn[row] = up / sqrtf(ss + p.l2_eps);
      if (row < 64) s.bad[row] = !finite(mx) || ss != ss;
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  if (tid == 0) {
    constexpr uint32_t idesc = idesc_f16(128, 64, false);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const uint64_t d = sdesc_k_sw128(smem_u32(s.kq[j >> 2])) + 2 * (j & 3);
      mma_bf16(tmem, d, d, idesc, j > 0);
    }
    mma_commit(&s.done);
    unsigned char* kq = c.kq + ((size_t)place * p.Hk + kh) * kq_bytes<D>();
#pragma unroll
    for (int a = 0; a < D / 64; ++a) {
      bulk_store(kq + a * 8192, s.kq[a], 8192);
      bulk_store(kq + (D / 64 + a) * 8192, s.kq[a] + 8192, 8192);
    }
    bulk_commit();
  }
  const int i = tid & 63;            // row of L (lanes 0..63) or of the causal products (64..127)
  const bool lower = (tid & 64) == 0;
  const int half = tid >> 7;         // columns 32 half ..
  bool ok = true;
  for (int g0 = 0; g0 < p.group; g0 += 2) {
    const int heads = min(2, p.group - g0);
    // gates: a warp for each head, two tokens a lane
    if (warp < heads) {
      const int h = kh * p.group + g0 + warp;
      const float rate = 1.4426950408889634f * expf(p.A_log[h]), shift = bf16_to_f(p.dt_bias[h]);
      float g[2], beta[2];
      int first_bad = 64;
#pragma unroll
      for (int k = 1; k >= 0; --k) {
        const int tok = 2 * lane + k;
        g[k] = beta[k] = 0.f;
        if (tok < n) {
          const __nv_bfloat16* ba = p.ba + (long long)(t0 + tok) * p.ldba;
          beta[k] = sigmoid_f(bf16_to_f(ba[h]));
          const float x = -rate * softplus_f(bf16_to_f(ba[p.Hv + h]) + shift);
          g[k] = x < -1e4f ? -1e4f : x;  // 2^-1e4 is 0, and sums of it stay ordinary
          if (!(finite(g[k]) && finite(beta[k])) || s.bad[tok]) first_bad = tok;
        }
      }
      Two a = add(Two{g[0], 0.f}, Two{g[1], 0.f});
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Two u{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
        if (lane >= o) a = add(u, a);
      }
      Two before{__shfl_up_sync(0xffffffffu, a.hi, 1), __shfl_up_sync(0xffffffffu, a.lo, 1)};
      if (lane == 0) before = Two{0.f, 0.f};
      const Two G[2] = {add(before, Two{g[0], 0.f}), a};
      const float ehi = __shfl_sync(0xffffffffu, a.hi, 31), elo = __shfl_sync(0xffffffffu, a.lo, 31);
      // of the last token of this lane's block of 16
      const float bhi = __shfl_sync(0xffffffffu, a.hi, lane | 7), blo = __shfl_sync(0xffffffffu, a.lo, lane | 7);
      float top = fmaxf(beta[0], beta[1]);
      for (int o = 16; o > 0; o >>= 1) {
        first_bad = min(first_bad, __shfl_xor_sync(0xffffffffu, first_bad, o));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int tok = 2 * lane + k;
        const float gam = exp2f(G[k].hi + G[k].lo), left = exp2f((ehi - G[k].hi) + (elo - G[k].lo));
        s.ghi[warp][tok] = G[k].hi;
        s.glo[warp][tok] = G[k].lo;
        s.bj[warp][tok] = s.rn[tok] * exp2f((bhi - G[k].hi) + (blo - G[k].lo));
        s.scal[warp][S_BETA][tok] = beta[k];
        s.scal[warp][S_C1][tok] = gam * s.rn[tok];
        s.scal[warp][S_CU][tok] = left * s.rn[tok];
        s.scal[warp][S_W][tok] = left * beta[k];
        s.scal[warp][S_CQG][tok] = p.q_scale * s.rn[64 + tok] * gam;
      }
      if (lane == 0) {
        s.scal[warp][S_END][0] = exp2f(ehi + elo);
        s.scal[warp][S_END][1] = __int_as_float(first_bad);
        s.scal[warp][S_END][2] = top;
      }
    }
    if (g0 == 0) {
      ok = mbar_wait(&s.done, 0);
      if (!ok) record(p.r.error, kStatusDeadline, kWhatWait, sq);
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // kq's room is free
    __syncthreads();
    tc_fence_after();
#pragma unroll 1
    for (int h = 0; h < heads; ++h) {
      // L_ij = beta_i e^(G_i-G_j) k_i.k_j and e^(G_i-G_j) q_i.k_j. Off the diagonal
      // blocks of 16, e^(G_i-G_j) is (from j to its block's end) x (from there to i),
      // both at most 1: one exponential a block and row.
      float dot[32];
      tmem_ld32(tmem + 32 * half + ((uint32_t)((warp & 3) * 32) << 16), dot);
      const float gi = s.ghi[h][i], li = s.glo[h][i];
      const float f = lower ? s.scal[h][S_BETA][i] * s.rn[i] : 1.f;
      float mx = 0.f;
#pragma unroll
      for (int jb = 0; jb < 2; ++jb) {
        const int j0 = 32 * half + 16 * jb;
        if (j0 > i) {
#pragma unroll
          for (int j = 0; j < 16; ++j) dot[16 * jb + j] = 0.f;
        } else if (j0 + 16 <= i) {
          const float a = f * exp2f((gi - s.ghi[h][j0 + 15]) + (li - s.glo[h][j0 + 15]));
#pragma unroll
          for (int j = 0; j < 16; ++j) dot[16 * jb + j] *= a * s.bj[h][j0 + j];
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int jj = j0 + j;
            const float x = f * s.rn[jj] * exp2f((gi - s.ghi[h][jj]) + (li - s.glo[h][jj])) * dot[16 * jb + j];
            dot[16 * jb + j] = jj < i || (jj == i && !lower) ? x : 0.f;
          }
        }
      }
      if (lower) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(s.m[h] + i * kLStride + 32 * half + j) = make_float4(dot[j], dot[j + 1], dot[j + 2], dot[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) mx = fmaxf(mx, fabsf(dot[j]));
        s.top[half][i] = mx;
      }
      __syncthreads();
      if (!lower) {
        // a row of the causal products takes a power of two of its own (S_CQ undoes it)
        const float f = row_scale(fmaxf(s.top[0][i], s.top[1][i]));
        if (half == 0) s.scal[h][S_CQ][i] = p.q_scale * s.rn[64 + i] * inverse_pow2(f);
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t w[4], wl[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) split2(make_float2(dot[j + 2 * k] * f, dot[j + 2 * k + 1] * f), &w[k], &wl[k]);
          *reinterpret_cast<uint4*>(s.a[h][0] + swz(i, 32 * half + j)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(s.a[h][1] + swz(i, 32 * half + j)) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
        }
      }
      __syncthreads();
    }
    // T = (I + L)^-1, in place of L. First its diagonal blocks of 16, a column a
    // thread: t_i = [i = col] - sum_{l < i} L_il t_l.
    const int hd = tid >> 7;  // the head this half of the threads works on
    if (tid < 64 * heads) {
      const int col = tid & 63, c16 = col & 15;
      float* L = s.m[tid >> 6] + (col & 48) * (kLStride + 1);
      float t[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float x0 = r == c16 ? 1.f : 0.f, x1 = 0.f;
#pragma unroll
        for (int l = 0; l < r; l += 4) {
          const float4 v = *reinterpret_cast<const float4*>(L + r * kLStride + l);
          x0 = fmaf(-v.x, t[l], x0);
          if (l + 1 < r) x1 = fmaf(-v.y, t[l + 1], x1);
          if (l + 2 < r) x0 = fmaf(-v.z, t[l + 2], x0);
          if (l + 3 < r) x1 = fmaf(-v.w, t[l + 3], x1);
        }
        t[r] = x0 + x1;
      }
      __syncwarp();  // a block's columns are one warp's: all have read it
#pragma unroll
      for (int r = 0; r < 16; ++r) L[r * kLStride + c16] = t[r];
    }
    __syncthreads();
    // Then twice the size at a time: [T11 0; L21 .] -> T21 = -T22 (L21 T11).
    {
      const int q = tid & 127, o = (q >> 6) * 32, r = (q & 63) >> 2, cc = (q & 3) * 4;
      float* m = s.m[hd] + o * (kLStride + 1);
      float* x = s.x[hd] + (q >> 6) * 16 * kXStride;
      if (hd < heads) {
        float4 v[1] = {};
        mac4(v, m + (16 + r) * kLStride, kLStride, m + cc, kLStride, 0, 16);
        *reinterpret_cast<float4*>(x + r * kXStride + cc) = v[0];
      }
      __syncthreads();
      if (hd < heads) {
        float4 v[1] = {};
        mac4(v, m + (16 + r) * kLStride + 16, kLStride, x + cc, kXStride, 0, 16);
        *reinterpret_cast<float4*>(m + (16 + r) * kLStride + cc) = minus(v[0]);
      }
      __syncthreads();
    }
    {
      const int q = tid & 127, r = (q >> 3) * 2, cc = (q & 7) * 4;
      float *m = s.m[hd], *x = s.x[hd];
      if (hd < heads) {
        float4 v[2] = {};
        mac4(v, m + (32 + r) * kLStride, kLStride, m + cc, kLStride, cc & 16, 32);  // T11 is 0 above its diagonal
        *reinterpret_cast<float4*>(x + r * kXStride + cc) = v[0];
        *reinterpret_cast<float4*>(x + (r + 1) * kXStride + cc) = v[1];
      }
      __syncthreads();
      if (hd < heads) {
        float4 v[2] = {};
        mac4(v, m + (32 + r) * kLStride + 32, kLStride, x + cc, kXStride, 0, (r & 16) + 16);  // and so is T22
        *reinterpret_cast<float4*>(m + (32 + r) * kLStride + cc) = minus(v[0]);
        *reinterpret_cast<float4*>(m + (33 + r) * kLStride + cc) = minus(v[1]);
      }
      __syncthreads();
    }
    if (hd < heads) {
#pragma unroll 2
      for (int q = tid & 127; q < 512; q += 128) {
        const int r = q >> 3, j = (q & 7) * 8;
        const float4 u = *reinterpret_cast<const float4*>(s.m[hd] + r * kLStride + j);
        const float4 v = *reinterpret_cast<const float4*>(s.m[hd] + r * kLStride + j + 4);
        uint32_t w[4], wl[4];
        split2(make_float2(u.x * kScaleT, u.y * kScaleT), &w[0], &wl[0]);
        split2(make_float2(u.z * kScaleT, u.w * kScaleT), &w[1], &wl[1]);
        split2(make_float2(v.x * kScaleT, v.y * kScaleT), &w[2], &wl[2]);
        split2(make_float2(v.z * kScaleT, v.w * kScaleT), &w[3], &wl[3]);
        *reinterpret_cast<uint4*>(s.t[hd][0] + swz(r, j)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(s.t[hd][1] + swz(r, j)) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      for (int h = 0; h < heads; ++h) {
        unsigned char* img = c.head + ((size_t)place * p.Hv + kh * p.group + g0 + h) * kHeadBytes;
        bulk_store(img, s.t[h][0], 16384);
        bulk_store(img + 16384, s.a[h][0], 16384);
        bulk_store(img + kImg, s.scal[h], S_COUNT * 256);
      }
      bulk_commit();
      if (g0 + 2 < p.group) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    __syncthreads();
  }
  if (tid == 0) bulk_wait_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 64);
}

// ------------------------------------------------------------------ the chunks of a sequence

// silu(z) before a rounding to bf16: the fast exponential and division (a few 2^-22)
// are far below it.
__device__ __forceinline__ float gate(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

constexpr int kChainThreads = 384;  // producer, MMA, TMEM, -; four warps of state rows; four of outputs

// TMEM columns
constexpr uint32_t kS = 0, kShi = 128, kSlo = 192, kPU = 256, kRhi = 320, kRlo = 352, kQS = 384, kAU = 448;
// U for the outputs, in the upper halves of S lo and S hi: what reads those is done
// when U is known
constexpr uint32_t kUhi = kSlo + 32, kUlo = kShi + 32;

template <int D>
struct alignas(1024) ChainStage {
  unsigned char k[64 * D * 2], q[64 * D * 2];  // f16 images
  unsigned char thi[8192], tlo[8192], ahi[8192], alo[8192];
  float scal[S_COUNT][64];
  __nv_bfloat16 v[64][D];
};

template <int D>
struct ChainSmem {
  ChainStage<D> st[2];
  float o[64][132];
  float inv_s[2][128], inv_u[2][128];
  int first_bad[2][128];
  uint64_t full[2], empty[2], s_ready[2], p_done, r_ready, u_done, u_ready, s_done[2], o_done, o_free, row_ready;
  uint32_t tmem;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kChainThreads, 1) delta_kernel(const ChunkParams c) {
  const DeltaParams& p = c.p;
  extern __shared__ unsigned char raw[];
  ChainSmem<D>& s = *reinterpret_cast<ChainSmem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x, sq = blockIdx.y, kh = h / p.group;
  int b, e, in, out;
  seq_rows(p.r, sq, &b, &e);
  if (e - b <= kRecurrentMax || !seq_slots(p.r, sq, false, &in, &out)) return;
  const int chunks = (e - b + kChunk - 1) / kChunk, place0 = chunk_first_place(p.r, sq);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 5);  // the MMA's commit and four output warps
      mbar_init(&s.s_ready[i], 4);
      mbar_init(&s.s_done[i], 1);
    }
    mbar_init(&s.p_done, 1);
    mbar_init(&s.r_ready, 4);
    mbar_init(&s.u_done, 1);
    mbar_init(&s.u_ready, 4);
    mbar_init(&s.o_done, 1);
    mbar_init(&s.o_free, 4);
    mbar_init(&s.row_ready, 4);
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc(&s.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  bool ok = true;

  if (warp == 0) {
    for (int n = 0; n < chunks; ++n) {
      const int t0 = b + n * kChunk, toks = min(kChunk, e - t0), st = n & 1;
      ChainStage<D>& g = s.st[st];
      ok = ok && mbar_wait(&s.empty[st], ((n >> 1) & 1) ^ 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const size_t place = place0 + n;
      if (lane == 0) {
        mbar_arrive_expect_tx(&s.full[st], kq_bytes<D>() + kHeadBytes + toks * D * 2);
        bulk_load(g.k, c.kq + (place * p.Hk + kh) * kq_bytes<D>(), kq_bytes<D>(), &s.full[st]);
        bulk_load(g.thi, c.head + (place * p.Hv + h) * kHeadBytes, kHeadBytes, &s.full[st]);
      }
      __syncwarp();
      for (int t = lane; t < toks; t += 32)
        bulk_load(g.v[t], p.qkv + (long long)(t0 + t) * p.ldqkv + 2 * p.Hk * D + h * D, D * 2, &s.full[st]);
    }
    // no copy is in flight when the CTA leaves
    for (int n = max(0, chunks - 2); n < chunks; ++n)
      if (ok) ok = mbar_wait(&s.full[n & 1], (n >> 1) & 1);
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_f16(128, 64, false), idesc_s = idesc_f16(128, 64, true);
    for (int n = 0; n < chunks && ok; ++n) {
      const int st = n & 1;
      const uint32_t ph = n & 1;
      ChainStage<D>& g = s.st[st];
      ok = mbar_wait(&s.full[st], (n >> 1) & 1);
      const uint32_t k = smem_u32(g.k), q = smem_u32(g.q);
      // P = S k, in halves of dk as they are ready
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        ok = ok && mbar_wait(&s.s_ready[hh], ph);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = hh * D / 32; j < (hh + 1) * D / 32; ++j) {
          const uint64_t bd = sdesc_k_sw128(k + (j >> 2) * 8192) + 2 * (j & 3);
          mma_f16_ts(tmem + kPU, tmem + kShi + 8 * j, bd, idesc, j > 0);
          mma_f16_ts(tmem + kPU, tmem + kSlo + 8 * j, bd, idesc, true);
        }
      }
      if (!ok) break;
      mma_commit(&s.p_done);
      // the state's part of the outputs, under the chain
      if (!(ok = mbar_wait(&s.o_free, ph ^ 1))) break;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const uint64_t bd = sdesc_k_sw128(q + (j >> 2) * 8192) + 2 * (j & 3);
        mma_f16_ts(tmem + kQS, tmem + kShi + 8 * j, bd, idesc, j > 0);
        mma_f16_ts(tmem + kQS, tmem + kSlo + 8 * j, bd, idesc, true);
      }
      // U = R T^T
      if (!(ok = mbar_wait(&s.r_ready, ph))) break;
      tc_fence_after();
      const uint64_t th = sdesc_k_sw128(smem_u32(g.thi)), tl = sdesc_k_sw128(smem_u32(g.tlo));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_f16_ts(tmem + kPU, tmem + kRhi + 8 * j, th + 2 * j, idesc, j > 0);
        mma_f16_ts(tmem + kPU, tmem + kRhi + 8 * j, tl + 2 * j, idesc, true);
        mma_f16_ts(tmem + kPU, tmem + kRlo + 8 * j, th + 2 * j, idesc, true);
      }
      mma_commit(&s.u_done);
      // S += U' k, 64 columns of dk at a time (U' hi, lo stand where R's were)
      if (!(ok = mbar_wait(&s.u_ready, ph))) break;
      tc_fence_after();
#pragma unroll
      for (int a = 0; a < D / 64; ++a) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t bd = sdesc_mn_sw128(k + a * 8192 + j * 2048, 8192);
          mma_f16_ts(tmem + kS + a * 64, tmem + kRhi + 8 * j, bd, idesc_s, true);
          mma_f16_ts(tmem + kS + a * 64, tmem + kRlo + 8 * j, bd, idesc_s, true);
        }
        mma_commit(&s.s_done[a]);
      }
      if (D == 64) mma_commit(&s.s_done[1]);
      const uint64_t ah = sdesc_k_sw128(smem_u32(g.ahi)), al = sdesc_k_sw128(smem_u32(g.alo));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_f16_ts(tmem + kAU, tmem + kUhi + 8 * j, ah + 2 * j, idesc, j > 0);
        mma_f16_ts(tmem + kAU, tmem + kUlo + 8 * j, ah + 2 * j, idesc, true);
        mma_f16_ts(tmem + kAU, tmem + kUhi + 8 * j, al + 2 * j, idesc, true);
      }
      mma_commit(&s.o_done);
      mma_commit(&s.empty[st]);
    }
    // no MMA is in flight when the TMEM is freed
    if (ok) ok = mbar_wait(&s.o_done, (chunks - 1) & 1);
  } else if (warp >= 4 && warp < 8) {
    // ---- the state's rows: thread = dv row
    const int row = tid - 128;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const bool real = row < D;
    // bound: of the row's 2-norm at the chunk's start, which fs is the scale of;
    // near: the same from the last measured norm
    float bound = 0.f, fs = 1.f;
    bool dead = false;  // the row holds a value that is not finite
    for (int pass = 0; pass < 2; ++pass) {
      // the starting state: its largest value, then the scaled accumulator
      float ss = 0.f, mx = 0.f;
      for (int col = 0; col < D; col += 32) {
        float x[32] = {};
        if (real && in > 0) {
          const size_t at = (((size_t)in * p.Hv + h) * D + row) * D + col;
          if constexpr (BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.state) + at + 8 * j);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) x[8 * j + 2 * k] = bf16_lo(w[k]), x[8 * j + 2 * k + 1] = bf16_hi(w[k]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.state) + at + 4 * j);
              x[4 * j] = v.x, x[4 * j + 1] = v.y, x[4 * j + 2] = v.z, x[4 * j + 3] = v.w;
            }
          }
        }
        if (pass == 0) {
#pragma unroll
          for (int j = 0; j < 32; ++j) mx = fmaxf(mx, fabsf(x[j])), ss += x[j] * 0.f;
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = dead ? 0.f : x[j] * fs;
          tmem_st32(tmem + kS + col + lanes, x);
        }
      }
      if (pass == 0) {
        dead = !(ss == 0.f);
        bound = dead ? 0.f : 12.f * mx;  // at least the 2-norm of 128 values
        fs = row_scale(bound);
      }
    }
    tmem_wait_st();
    float near = bound;
    for (int n = 0; n < chunks; ++n) {
      const int st = n & 1, toks = min(kChunk, e - (b + n * kChunk));
      const uint32_t ph = n & 1;
      ChainStage<D>& g = s.st[st];
      if (ok) ok = mbar_wait(&s.full[st], (n >> 1) & 1);
      // This row's v over the chunk, zero past the sequence's end. (The lanes past D
      // = 64 rows do as those of the first 64, from a zero state; nobody reads them.)
      uint32_t v[32];
      {
        const __nv_bfloat16* vr = &g.v[0][row & (D - 1)];
#pragma unroll
        for (int i = 0; i < 32; ++i)
          v[i] = __bfloat16_as_ushort(vr[2 * i * D]) | ((uint32_t)__bfloat16_as_ushort(vr[(2 * i + 1) * D]) << 16);
      }
      if (toks < kChunk) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] &= 2 * i + 1 < toks ? 0xffffffffu : 2 * i < toks ? 0xffffu : 0u;
      }
      // sums of beta |v| and of e^(G_C-G) beta |v|, the largest |v|
      int first_bad = __float_as_int(g.scal[S_END][1]);
      float sb, sw, mv;
      const auto sums = [&]() {
        float2 b2 = make_float2(0.f, 0.f), w2 = b2;
        float m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float4 be = *reinterpret_cast<const float4*>(&g.scal[S_BETA][i]);
          const float4 w = *reinterpret_cast<const float4*>(&g.scal[S_W][i]);
          const uint32_t p0 = v[i / 2] & 0x7fff7fffu, p1 = v[i / 2 + 1] & 0x7fff7fffu;
          const float2 a0 = make_float2(bf16_lo(p0), bf16_hi(p0)), a1 = make_float2(bf16_lo(p1), bf16_hi(p1));
          b2 = __ffma2_rn(make_float2(be.x, be.y), a0, b2);
          w2 = __ffma2_rn(make_float2(w.x, w.y), a0, w2);
          b2 = __ffma2_rn(make_float2(be.z, be.w), a1, b2);
          w2 = __ffma2_rn(make_float2(w.z, w.w), a1, w2);
          m0 = fmaxf(m0, fmaxf(a0.x, a0.y));
          m1 = fmaxf(m1, fmaxf(a1.x, a1.y));
        }
        sb = b2.x + b2.y, sw = w2.x + w2.y, mv = fmaxf(m0, m1);
      };
      sums();
      float gam_end = g.scal[S_END][0];
      if (first_bad < 64 || !finite(sb)) {
        // a row that stops being finite: zeros from there on
#pragma unroll
        for (int i = 31; i >= 0; --i) {
          if (!finite(bf16_hi(v[i]))) first_bad = min(first_bad, 2 * i + 1);
          if (!finite(bf16_lo(v[i]))) first_bad = min(first_bad, 2 * i);
        }
        sb = mv = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          v[i] &= 2 * i + 1 < first_bad ? 0xffffffffu : 2 * i < first_bad ? 0xffffu : 0u;
          const float a = fmaxf(fabsf(bf16_lo(v[i])), fabsf(bf16_hi(v[i])));
          sb += 2.f * a;  // beta <= 1
          mv = fmaxf(mv, a);
        }
        gam_end = sw = 0.f;
      }
      if (dead) first_bad = 0;
      // scales: of U, and of the state after this chunk
      const float fu = row_scale((first_bad < 64 ? 1.f : g.scal[S_END][2]) * (mv + bound + sb));
      bound = fmaf(gam_end, fminf(bound, near), sw) * 1.01f;
      const float fs_next = row_scale(bound);
      const float shrink = gam_end * fminf(fs_next * inverse_pow2(fs), 0x1p126f);
      float2 ss2 = make_float2(0.f, 0.f);
      const float2 shrink2 = make_float2(shrink, shrink);
#pragma unroll 1
      for (int col = 0; col < D; col += 32) {
        const int hh = col >= D / 2;
        if (n > 0 && (col & (D / 2 - 1)) == 0) {
          if (ok) ok = mbar_wait(&s.s_done[hh], ph ^ 1);
          if (hh == 1 && ok) ok = mbar_wait(&s.o_done, ph ^ 1);  // U stood in the upper halves
          tc_fence_after();
        }
        float x[32];
        uint32_t hi[16], lo[16];
        tmem_ld32(tmem + kS + col + lanes, x);
        if (dead) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 y = make_float2(x[j], x[j + 1]);
          ss2 = __ffma2_rn(y, y, ss2);
          split2(y, &hi[j / 2], &lo[j / 2]);
          const float2 z = __fmul2_rn(y, shrink2);
          x[j] = z.x, x[j + 1] = z.y;
        }
        tmem_st16(tmem + kShi + col / 2 + lanes, hi);
        tmem_st16(tmem + kSlo + col / 2 + lanes, lo);
        tmem_st32(tmem + kS + col + lanes, x);
        if ((col & (D / 2 - 1)) == D / 2 - 32) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.s_ready[hh]);
        }
      }
      const float ss = ss2.x + ss2.y;
      const float inv_s = inverse_pow2(fs), p_scale = fminf(fu * inv_s, 0x1p126f);
      near = fmaf(gam_end, sqrtf(ss) * inv_s, sw) * 1.01f;
      s.inv_s[st][row] = inv_s;
      s.inv_u[st][row] = inverse_pow2(fu);
      s.first_bad[st][row] = first_bad;
      if (ok) ok = mbar_wait(&s.p_done, ph);
      tc_fence_after();
      // zeros from the first token on that is past the end or not finite
      const int until = min(first_bad, toks);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[32];
        uint32_t hi[16], lo[16];
        tmem_ld32(tmem + kPU + half * 32 + lanes, x);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const int i = half * 32 + j;
          const float4 be = *reinterpret_cast<const float4*>(&g.scal[S_BETA][i]);
          const float4 c1 = *reinterpret_cast<const float4*>(&g.scal[S_C1][i]);
          const float2 f2 = make_float2(fu, fu), p2 = make_float2(-p_scale, -p_scale);
          const float2 v0 = make_float2(bf16_lo(v[i / 2]), bf16_hi(v[i / 2]));
          const float2 v1 = make_float2(bf16_lo(v[i / 2 + 1]), bf16_hi(v[i / 2 + 1]));
          const float2 q0 = __fmul2_rn(__fmul2_rn(make_float2(x[j], x[j + 1]), p2), make_float2(c1.x, c1.y));
          const float2 q1 = __fmul2_rn(__fmul2_rn(make_float2(x[j + 2], x[j + 3]), p2), make_float2(c1.z, c1.w));
          float2 r0 = __fmul2_rn(make_float2(be.x, be.y), __ffma2_rn(f2, v0, q0));
          float2 r1 = __fmul2_rn(make_float2(be.z, be.w), __ffma2_rn(f2, v1, q1));
          if (until < 64) {
            if (i >= until) r0.x = 0.f;
            if (i + 1 >= until) r0.y = 0.f;
            if (i + 2 >= until) r1.x = 0.f;
            if (i + 3 >= until) r1.y = 0.f;
          }
          split2(r0, &hi[j / 2], &lo[j / 2]);
          split2(r1, &hi[j / 2 + 1], &lo[j / 2 + 1]);
        }
        tmem_st16(tmem + kRhi + half * 16 + lanes, hi);
        tmem_st16(tmem + kRlo + half * 16 + lanes, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.r_ready);
      const float u_scale = fminf(fs_next * inverse_pow2(fu), 0x1p126f);
      if (ok) ok = mbar_wait(&s.u_done, ph);
      tc_fence_after();
      const float2 us2 = make_float2(u_scale, u_scale), t2 = make_float2(1.0f / kScaleT, 1.0f / kScaleT);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        float u[32];
        uint32_t hi[16], lo[16], ohi[16], olo[16];
        tmem_ld32(tmem + kPU + half * 32 + lanes, u);
        if (first_bad < 64) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (half * 32 + j >= first_bad) u[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 cu = *reinterpret_cast<const float4*>(&g.scal[S_CU][half * 32 + j]);
          const float2 cs[2] = {make_float2(cu.x, cu.y), make_float2(cu.z, cu.w)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 y = __fmul2_rn(make_float2(u[j + 2 * k], u[j + 2 * k + 1]), t2);
            split2(y, &ohi[j / 2 + k], &olo[j / 2 + k]);
            float2 w = __fmul2_rn(__fmul2_rn(y, us2), cs[k]);
            if (first_bad < 64) w = make_float2(0.f, 0.f);
            split2(w, &hi[j / 2 + k], &lo[j / 2 + k]);
          }
        }
        tmem_st16(tmem + kRhi + half * 16 + lanes, hi);
        tmem_st16(tmem + kRlo + half * 16 + lanes, lo);
        tmem_st16(tmem + kUhi + half * 16 + lanes, ohi);
        tmem_st16(tmem + kUlo + half * 16 + lanes, olo);
      }
      if (first_bad < 64) dead = true;
      fs = fs_next;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      // row_ready goes with u_ready, not before: this chunk's U waited for the
      // outputs of the chunk before (o_free), so row_ready never runs two phases
      // ahead of the output warps
      if (lane == 0) {
        mbar_arrive(&s.u_ready);
        mbar_arrive(&s.row_ready);
      }
    }
    // the state after the last chunk
    const uint32_t ph = (chunks - 1) & 1;
    if (ok) ok = mbar_wait(&s.s_done[0], ph);
    if (ok) ok = mbar_wait(&s.s_done[1], ph);
    tc_fence_after();
    const float nan = __int_as_float(0x7fffffff), inv = inverse_pow2(fs);
    for (int col = 0; col < D; col += 32) {
      float x[32];
      tmem_ld32(tmem + kS + col + lanes, x);
      if (!real || !ok) continue;
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = dead ? nan : x[j] * inv;
      const size_t at = (((size_t)out * p.Hv + h) * D + row) * D + col;
      if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.state) + at + 8 * j) =
              make_uint4(pack_bf16x2(x[8 * j], x[8 * j + 1]), pack_bf16x2(x[8 * j + 2], x[8 * j + 3]),
                         pack_bf16x2(x[8 * j + 4], x[8 * j + 5]), pack_bf16x2(x[8 * j + 6], x[8 * j + 7]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(static_cast<float*>(p.state) + at + 4 * j) =
              make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      }
    }
  } else if (warp >= 8) {
    // ---- the outputs
    const int row = tid - 256, w = warp - 8;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // On the way out eight lanes take a row, four columns in every 32 each; a warp
    // the rows 16 w .. 16 w + 15, four at a time.
    constexpr int E = D / 32;
    const int sub = lane >> 3, l8 = (lane & 7) * 4;
    float gw[E][4] = {};
    if (p.z) {
#pragma unroll
      for (int k = 0; k < E; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) gw[k][j] = bf16_to_f(p.gnorm_w[32 * k + l8 + j]);
    }
    for (int n = 0; n < chunks; ++n) {
      const int st = n & 1, t0 = b + n * kChunk, toks = min(kChunk, e - t0);
      const uint32_t ph = n & 1;
      ChainStage<D>& g = s.st[st];
      // this warp's rows of z, in flight while the chunk is finished
      uint2 z[4][E];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * w + 4 * i + sub;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          z[i][k] = make_uint2(0, 0);
          if (p.z && t < toks)
            z[i][k] = __ldg(reinterpret_cast<const uint2*>(p.z + (long long)(t0 + t) * p.ldz + h * D + 32 * k + l8));
        }
      }
      if (ok) ok = mbar_wait(&s.row_ready, ph);
      if (ok) ok = mbar_wait(&s.full[st], (n >> 1) & 1);
      const float inv_s = s.inv_s[st][row], inv_u = s.inv_u[st][row];
      const int first_bad = s.first_bad[st][row];
      if (ok) ok = mbar_wait(&s.o_done, ph);
      tc_fence_after();
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        float x[32], y[32];
        tmem_ld32(tmem + kQS + half * 32 + lanes, x);
        tmem_ld32(tmem + kAU + half * 32 + lanes, y);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const int i = half * 32 + j;
          const float4 cg = *reinterpret_cast<const float4*>(&g.scal[S_CQG][i]);
          const float4 cq = *reinterpret_cast<const float4*>(&g.scal[S_CQ][i]);
          s.o[i][row] = fmaf(cg.x, x[j] * inv_s, cq.x * (y[j] * inv_u));
          s.o[i + 1][row] = fmaf(cg.y, x[j + 1] * inv_s, cq.y * (y[j + 1] * inv_u));
          s.o[i + 2][row] = fmaf(cg.z, x[j + 2] * inv_s, cq.z * (y[j + 2] * inv_u));
          s.o[i + 3][row] = fmaf(cg.w, x[j + 3] * inv_s, cq.w * (y[j + 3] * inv_u));
        }
      }
      for (int i = first_bad; i < kChunk; ++i) s.o[i][row] = __int_as_float(0x7fffffff);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.o_free);
        mbar_arrive(&s.empty[st]);
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");  // the output warps: every row is staged
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * w + 4 * i + sub;
        float4 o[E];
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] = *reinterpret_cast<const float4*>(&s.o[t][32 * k + l8]);
        if (p.z) {
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < E; ++k)
            sum = fmaf(o[k].x, o[k].x, fmaf(o[k].y, o[k].y, fmaf(o[k].z, o[k].z, fmaf(o[k].w, o[k].w, sum))));
#pragma unroll
          for (int m = 4; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
          const float r = rsqrtf(sum * (1.0f / D) + p.gnorm_eps);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float zf[4] = {bf16_lo(z[i][k].x), bf16_hi(z[i][k].x), bf16_lo(z[i][k].y), bf16_hi(z[i][k].y)};
            o[k].x *= r * gw[k][0] * gate(zf[0]);
            o[k].y *= r * gw[k][1] * gate(zf[1]);
            o[k].z *= r * gw[k][2] * gate(zf[2]);
            o[k].w *= r * gw[k][3] * gate(zf[3]);
          }
        }
        if (t < toks) {
          __nv_bfloat16* dst = p.out + (long long)(t0 + t) * p.ldo + h * D + l8;
#pragma unroll
          for (int k = 0; k < E; ++k)
            *reinterpret_cast<uint2*>(dst + 32 * k) = make_uint2(pack_bf16x2(o[k].x, o[k].y), pack_bf16x2(o[k].z, o[k].w));
        }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");  // before the next chunk is staged
    }
  }
  if (!ok) record(p.r.error, kStatusDeadline, kWhatWait, sq);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host

template <auto* KERNEL>
cudaError_t opt_in(size_t bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t f = cudaFuncSetAttribute((const void*)KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (f == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return f;
}

template <int D, bool BF16>
cudaError_t launch(const ChunkParams& c, cudaStream_t s) {
  const size_t prep = sizeof(PrepSmem<D>) + 1024, chain = sizeof(ChainSmem<D>) + 1024;
  static_assert(sizeof(ChainSmem<D>) + 1024 <= 232448, "227 KB of shared memory a CTA");
  cudaError_t e = opt_in<prepare_kernel<D>>(prep);
  if (e == cudaSuccess) e = opt_in<delta_kernel<D, BF16>>(chain);
  if (e != cudaSuccess) return e;
  const dim3 places(chunk_places(c.p.r.tokens, c.p.r.seqs) - 1, c.p.Hk);  // the last is the pad rows'
  prepare_kernel<D><<<places, kPrepThreads, prep, s>>>(c);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  delta_kernel<D, BF16><<<dim3(c.p.Hv, c.p.r.seqs), kChainThreads, chain, s>>>(c);
  return cudaGetLastError();
}

}  // namespace

size_t delta_chunk_bytes(long long tokens, long long seqs, int Hk, int Hv, int d) {
  const size_t places = (size_t)(tokens / kChunk + seqs + 1);
  return places * ((size_t)Hk * 2 * kChunk * d * 2 + (size_t)Hv * kHeadBytes);
}

cudaError_t launch_delta_chunks(const DeltaParams& p, int d, bool state_bf16, unsigned char* ws, cudaStream_t s) {
  ChunkParams c;
  c.p = p;
  c.kq = ws;
  c.head = ws + (size_t)chunk_places(p.r.tokens, p.r.seqs) * p.Hk * 2 * kChunk * d * 2;
  if (d == 128) return state_bf16 ? launch<128, true>(c, s) : launch<128, false>(c, s);
  return state_bf16 ? launch<64, true>(c, s) : launch<64, false>(c, s);
}

}  // namespace gdn
