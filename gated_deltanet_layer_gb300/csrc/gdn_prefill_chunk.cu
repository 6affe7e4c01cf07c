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
//   |u_j|, |R_j| <= max(beta) (max |v| + sum beta |v|) + max(e^G beta) |S0|,
// with the row's largest |v| of the chunk for every |v|, and its norm measured every eighth
// chunk; |T| <= 1 takes the constant 2^12. Two terms reach 2^-39 of such a bound, which no
// other row's values are part of.
//
// What bounds it. One chunk follows the other: a sequence's chunk takes 3.2 us (2916
// tokens on one rank's shard: 152 us for 46), of which the three dependent products are
// about 0.9 and the conversions of S, R and U to f16 between them the rest; the tensor
// pipe is 30% busy, an SM issues every second cycle. A CTA's start and end take 9 us
// beside its chunks. 13 sequences of 16384 tokens on 64 heads take 359 us, 16700 chunks on
// 152 SMs, and 1.35 GB from and to memory (3.7 TB/s), of which the images are half.
// prepare_kernel takes 28 us for one round of CTAs and 291 for those 16384 tokens; it is
// bound by its instructions (an SM issues half of its slots) between short steps that wait
// for one another, and moves 0.70 GB (2.4 TB/s), the images it writes being 0.55.
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
// A chunk's images and scalars of a value head, arrays of 64 floats: what the state's
// chain needs (T hi, T lo) and what the outputs need (causal products hi, lo).
// S_R: of every two tokens beta, beta, c, c with c = e^G / |k|; S_CU:
// e^(G_C-G) / |k|; S_END: see below.
enum { S_R = 0, S_CU = 2, S_END, S_COUNT };
enum { O_CQG, O_CQ, O_COUNT };
constexpr int kImg = 2 * 8192;  // two images of 64 x 64 f16
constexpr int kChainBytes = kImg + S_COUNT * 256, kOutBytes = kImg + O_COUNT * 256;
constexpr int kHeadBytes = kChainBytes + kOutBytes;
// S_END: [0] e^(G_C), [1] (an int) the first token whose k or gates are not finite,
// else 64, [2] the largest beta, [3] sum beta, [4] sum e^(G_C-G) beta, [5] the largest
// e^G beta.

template <int D>
constexpr int kq_bytes() { return 2 * kChunk * D * 2; }  // the k image, then q's

struct ChunkParams {
  DeltaParams p;
  unsigned char* kq;    // [place][Hk] f16 images of k and q
  unsigned char* head;  // [place][Hv] images and scalars
  int ahead;            // prepare CTAs that run at once
};

// Byte of (row, column) in a K-major operand image of 64 f16 columns, 128-byte swizzle.
__device__ __forceinline__ int swz(int row, int col) { return row * 128 + ((((col >> 3) ^ row) & 7) << 4) + (col & 7) * 2; }

__device__ __forceinline__ uint32_t pack_h2(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// y = hi + lo, two f16 each: hi is y rounded to f16's 11 bits, and what is left is exact, by
// a multiply-add that takes the f16 itself. (An instruction in ten fewer than with y cut
// and subtracted in f32: 13 sequences, 16384 tokens 411 -> 395 us.)
__device__ __forceinline__ void split2(float2 y, uint32_t* hi, uint32_t* lo) {
  const uint32_t h = pack_h2(__float22half2_rn(y));
  float2 d;
  asm("{\n\t.reg .b16 a, b, m;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "mov.b16 m, 0xBC00;\n\t"
      "fma.rn.f32.f16 %0, a, m, %3;\n\t"
      "fma.rn.f32.f16 %1, b, m, %4;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(h), "f"(y.x), "f"(y.y));
  *hi = h;
  *lo = pack_h2(__float22half2_rn(d));
}

// v f + q for two bf16 v and a bf16 f.
__device__ __forceinline__ float2 add_scaled(uint32_t v, uint16_t f, float2 q) {
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "fma.rn.f32.bf16 %0, a, %3, %4;\n\t"
      "fma.rn.f32.bf16 %1, b, %3, %5;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v), "h"(f), "f"(q.x), "f"(q.y));
  return r;
}

// 16 columns (a multiple of 16 on) of a row of such an image: the swizzle keeps the two
// 16-byte pieces in one aligned 32 bytes, the second first in odd rows.
__device__ __forceinline__ void store_pair(unsigned char* image, int row, int col, const uint32_t (&w)[8]) {
  const bool odd = row & 1;
  unsigned char* p = image + (swz(row, col) & ~31);
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(odd ? w[4] : w[0]), "r"(odd ? w[5] : w[1]),
               "r"(odd ? w[6] : w[2]), "r"(odd ? w[7] : w[3]), "r"(odd ? w[0] : w[4]), "r"(odd ? w[1] : w[5]),
               "r"(odd ? w[2] : w[6]), "r"(odd ? w[3] : w[7])
               : "memory");
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
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16f(uint32_t t, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  tmem_st16(t, r);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A bound past the largest float is the largest: infinity x a gate of 0 would be no bound.
// For the same reason a scale that takes a power of two back multiplies last, after the
// gates.
constexpr float kLargest = 0x1.fffffep127f;

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

// A CTA takes a chunk of one key head and four of its value heads at once, 128 threads
// each, which meet at barriers of their own: every step is short and waits on the one
// before, so heads side by side (and two CTAs an SM) are what fills the time.
constexpr int kPrepHeads = 4;
constexpr int kPrepThreads = 128 * kPrepHeads;
constexpr int kLStride = 68;  // floats of a row of L: 16-byte rows, apart in banks
constexpr int kXStride = 36;

template <int D>
struct alignas(1024) PrepSmem {
  union {
    unsigned char kq[D / 64][128 * 128];     // rows k 0..63, q 0..63, in atoms of 64 columns
    float x[kPrepHeads][32 * kXStride];      // later a product on T's way
  };
  float m[kPrepHeads][64 * kLStride];        // L, then T in its place
  float ghi[kPrepHeads][64], glo[kPrepHeads][64];  // running sums of the log2 gates
  float bj[kPrepHeads][64];                  // 2^(G of the 16-block's end - G_j) / |k_j|
  int steep[kPrepHeads][4];                  // a block's gates fall by more than 2^100
  int first_bad[kPrepHeads];                 // first token whose k or gates are not finite, else 64
  float beta[kPrepHeads][64];
  float rn[128];                             // 1 / norm of the f16 rows (k, q)
  int bad[64];                               // k not finite
  uint64_t done;
  uint32_t tmem;
};

// x[i] += sum_l A[i][l] B[l][c..c+3] for R rows i of A, l0 <= l < l1 (multiples of 4).
template <int R>
__device__ __forceinline__ void mac4(float4 (&x)[R], const float* A, int lda, const float* B, int ldb, int l0, int l1) {
#pragma unroll 2
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
  // The delta kernel may take an SM as soon as no CTA of this one is left to start.
  griddep_launch_dependents();
  const DeltaParams& p = c.p;
  extern __shared__ unsigned char raw[];
  PrepSmem<D>& s = *reinterpret_cast<PrepSmem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int place = blockIdx.x / p.Hk, kh = blockIdx.x % p.Hk, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int b, e;
  const int sq = chunk_seq<false>(p.r, place, &b, &e);
  const int t0 = b + (place - chunk_first_place(sq, b)) * kChunk, n = min(kChunk, e - t0);
  if (n <= 0 || e - b <= kRecurrentMax || !seq_live(p.r, sq, seq_in(p.r, sq), b, e, false)) {
    griddep_wait();
    return;
  }
  // k and q rows: norms, and f16 images scaled by a power of two each
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIter = 128 / (kPrepThreads / 32) / kRows;
  uint4 row_in[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int row = (warp * kIter + i) * kRows + lane / kLanes, tok = row & 63, col = (lane % kLanes) * 8;
    row_in[i] = make_uint4(0, 0, 0, 0);
    if (tok < n)
      row_in[i] = __ldg(reinterpret_cast<const uint4*>(p.qkv + (long long)(t0 + tok) * p.ldqkv + (row < 64 ? p.Hk + kh : kh) * D + col));
  }
  // The rows of the CTA that will follow this one on its SM, two CTAs an SM, into L2:
  // k and q come from memory, and nothing else is there to do meanwhile.
  {
    const long long ahead = (long long)t0 + (c.ahead + p.Hk - 1) / p.Hk * kChunk + (tid >> 3 & 63);
    const int part = (tid & 7) * 64;  // 128 bytes of k's D columns (the first lanes), then of q's
    if (tid < 512 && part < 2 * D && ahead < p.r.tokens)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.qkv + ahead * p.ldqkv + (part < D ? (p.Hk + kh) * D + part : kh * D + part - D)));
  }
  // and what the first heads' gates are made of
  const int hd = tid >> 7, q = tid & 127;  // this thread's head of the four, and its place in it
  float gate_in[2][2] = {}, gate_w[2] = {};
  const auto load_gates = [&](int h) {
    gate_w[0] = p.A_log[h], gate_w[1] = bf16_to_f(p.dt_bias[h]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (2 * lane + k < n) {
        const __nv_bfloat16* ba = p.ba + (long long)(t0 + 2 * lane + k) * p.ldba;
        gate_in[k][0] = bf16_to_f(ba[h]), gate_in[k][1] = bf16_to_f(ba[p.Hv + h]);
      }
  };
  if (q < 32 && hd < p.group) load_gates(kh * p.group + hd);
  if (warp == 0) tmem_alloc(&s.tmem, 64);
  if (tid == 0) {
    mbar_init(&s.done, 1);
    fence_mbar_init();
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int row = (warp * kIter + i) * kRows + lane / kLanes, col = (lane % kLanes) * 8;
    const uint32_t w[4] = {row_in[i].x, row_in[i].y, row_in[i].z, row_in[i].w};
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
      // Without an l2_eps a zero row has no norm: a key's token is then one that is not
      // finite. Rows past the last token are zeros of nobody's.
      const float rn = (row & 63) < n ? up / sqrtf(ss + p.l2_eps) : 0.f;
      s.rn[row] = rn;
      if (row < 64) s.bad[row] = !finite(mx) || ss != ss || !finite(rn);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  constexpr int kStoreWarp = kPrepThreads / 32 - 1;
  if (warp == 1 && elect_one()) {
    constexpr uint32_t idesc = idesc_f16(128, 64, false);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const uint64_t d = sdesc_k_sw128(smem_u32(s.kq[j >> 2])) + 2 * (j & 3);
      mma_bf16(tmem, d, d, idesc, j > 0);
    }
    mma_commit(&s.done);
  }
  if (warp == kStoreWarp && lane == 0) {
    unsigned char* kq = c.kq + ((size_t)place * p.Hk + kh) * kq_bytes<D>();
#pragma unroll
    for (int a = 0; a < D / 64; ++a) {
      bulk_store(kq + a * 8192, s.kq[a], 8192);
      bulk_store(kq + (D / 64 + a) * 8192, s.kq[a] + 8192, 8192);
    }
    bulk_commit();
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the room is x's below
  }
  __syncwarp();
  const int i = q & 63;                    // row of L (TMEM lanes 0..63) or of the causal products (64..127)
  const bool lower = q < 64;
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + hd) : "memory"); };
  bool ok = true;
  for (int g0 = 0; g0 < p.group; g0 += kPrepHeads) {
    const int g = g0 + hd, h = kh * p.group + g;
    const bool mine = g < p.group;
    unsigned char* img = c.head + ((size_t)place * p.Hv + h) * kHeadBytes;
    // gates: one warp a head, two tokens a lane
    if (q < 32 && mine) {
      if (g0 > 0) load_gates(h);
      const float rate = 1.4426950408889634f * expf(gate_w[0]), shift = gate_w[1];
      float gt[2], beta[2];
      int first_bad = 64;
#pragma unroll
      for (int k = 1; k >= 0; --k) {
        const int tok = 2 * lane + k;
        gt[k] = beta[k] = 0.f;
        if (tok < n) {
          beta[k] = sigmoid_f(gate_in[k][0]);
          const float x = -rate * softplus_f(gate_in[k][1] + shift);
          gt[k] = x < -1e4f ? -1e4f : x;  // 2^-1e4 is 0, and sums of it stay ordinary
          if (!(finite(gt[k]) && finite(beta[k])) || s.bad[tok]) first_bad = tok;
        }
      }
      Two a = add(Two{gt[0], 0.f}, Two{gt[1], 0.f});
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Two u{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
        if (lane >= o) a = add(u, a);
      }
      Two before{__shfl_up_sync(0xffffffffu, a.hi, 1), __shfl_up_sync(0xffffffffu, a.lo, 1)};
      if (lane == 0) before = Two{0.f, 0.f};
      const Two G[2] = {add(before, Two{gt[0], 0.f}), a};
      const float ehi = __shfl_sync(0xffffffffu, a.hi, 31), elo = __shfl_sync(0xffffffffu, a.lo, 31);
      // of the last token of this lane's block of 16
      const float bhi = __shfl_sync(0xffffffffu, a.hi, lane | 7), blo = __shfl_sync(0xffffffffu, a.lo, lane | 7);
      first_bad = __reduce_min_sync(0xffffffffu, first_bad);
      const auto largest = [](float a, float b) {  // of values that are not negative: as their bits
        return __uint_as_float(__reduce_max_sync(0xffffffffu, max(__float_as_uint(a), __float_as_uint(b))));
      };
      if ((lane & 7) == 0) s.steep[hd][lane >> 3] = !(G[0].hi - bhi < 100.f);
      float gam[2], left[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int tok = 2 * lane + k;
        gam[k] = exp2f(G[k].hi + G[k].lo), left[k] = exp2f((ehi - G[k].hi) + (elo - G[k].lo));
        s.ghi[hd][tok] = G[k].hi;
        s.glo[hd][tok] = G[k].lo;
        s.bj[hd][tok] = s.rn[tok] * exp2f((bhi - G[k].hi) + (blo - G[k].lo));
        s.beta[hd][tok] = beta[k];
      }
      const float2 rn = *reinterpret_cast<const float2*>(&s.rn[2 * lane]), rq = *reinterpret_cast<const float2*>(&s.rn[64 + 2 * lane]);
      float* sc = reinterpret_cast<float*>(img + kImg);
      *reinterpret_cast<float4*>(sc + 64 * S_R + 4 * lane) =
          make_float4(beta[0], beta[1], gam[0] * rn.x, gam[1] * rn.y);
      *reinterpret_cast<float2*>(sc + 64 * S_CU + 2 * lane) = make_float2(left[0] * rn.x, left[1] * rn.y);
      const float sum_b = warp_sum(beta[0] + beta[1]), sum_w = warp_sum(left[0] * beta[0] + left[1] * beta[1]);
      const float top = largest(beta[0], beta[1]), reach = largest(beta[0] * gam[0], beta[1] * gam[1]);
      if (lane == 0) {
        *reinterpret_cast<float4*>(sc + 64 * S_END) = make_float4(exp2f(ehi + elo), __int_as_float(first_bad), top, sum_b);
        *reinterpret_cast<float2*>(sc + 64 * S_END + 4) = make_float2(sum_w, reach);
        s.first_bad[hd] = first_bad;
      }
      *reinterpret_cast<float2*>(img + kChainBytes + kImg + 256 * O_CQG + 8 * lane) =
          make_float2(p.q_scale * rq.x * gam[0], p.q_scale * rq.y * gam[1]);
    }
    if (g0 == 0) {
      ok = mbar_wait(&s.done, 0);
      if (!ok) record(p.r.error, kStatusDeadline, kWhatWait, sq);
      __syncthreads();  // and kq is read out
      tc_fence_after();
    } else {
      meet();
    }
    if (!mine) continue;  // a whole head's threads
    // L_ij = beta_i e^(G_i-G_j) k_i.k_j and e^(G_i-G_j) q_i.k_j, 16 columns at a time:
    // e^(G_i-G_j) is (from j to its block's end) x (from there to i), one exponential a
    // block and row. Both are at most 1 but on the diagonal, where the second undoes up
    // to the block's whole fall; a block that falls by more than 2^100 takes an
    // exponential a value there.
    const float gi = s.ghi[hd][i], li = s.glo[hd][i];
    const float f = lower ? s.beta[hd][i] * s.rn[i] : 1.f;
    const int until = lower ? i : i + 1;
    const auto block = [&](int j0, float (&x)[16]) {
      tmem_ld16(tmem + j0 + lanes, x);
      if (s.steep[hd][j0 >> 4] && j0 <= i && i < j0 + 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int jj = j0 + j;
          x[j] *= f * s.rn[jj] * exp2f(jj <= i ? (gi - s.ghi[hd][jj]) + (li - s.glo[hd][jj]) : 0.f);
        }
      } else {
        const float a = j0 > i ? 0.f : f * exp2f((gi - s.ghi[hd][j0 + 15]) + (li - s.glo[hd][j0 + 15]));
        const float2 a2 = make_float2(a, a);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 bj = *reinterpret_cast<const float4*>(&s.bj[hd][j0 + j]);
          const float2 y0 = __fmul2_rn(make_float2(x[j], x[j + 1]), __fmul2_rn(a2, make_float2(bj.x, bj.y)));
          const float2 y1 = __fmul2_rn(make_float2(x[j + 2], x[j + 3]), __fmul2_rn(a2, make_float2(bj.z, bj.w)));
          x[j] = y0.x, x[j + 1] = y0.y, x[j + 2] = y1.x, x[j + 3] = y1.y;
        }
      }
      if (j0 + 16 > (i & 32)) {  // the warp's rows cross the diagonal here
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j0 + j >= until) x[j] = 0.f;
      }
    };
    const int last = i & 32 ? 64 : 32;  // this warp's rows end before this column
    if (lower) {
#pragma unroll 1
      for (int j0 = 0; j0 < last; j0 += 16) {
        float x[16];
        block(j0, x);
        // U is zero from the first token on that is not finite; so is L, or its NaN
        // would reach earlier rows of T through products with T's zeros
        if (i >= s.first_bad[hd]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(s.m[hd] + i * kLStride + j0 + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
      }
      asm volatile("bar.sync %0, 64;" ::"r"(5 + hd) : "memory");  // the two warps of L
    } else {
      // The causal products, a row at a power of two of its own (O_CQ undoes it), while
      // the other two warps begin on T.
      float mx = 0.f;
#pragma unroll 1
      for (int j0 = 0; j0 < last; j0 += 16) {
        float x[16];
        block(j0, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) mx = fmaxf(mx, fabsf(x[j]));
      }
      const float fa = row_scale(mx);
      unsigned char* a = img + kChainBytes;
      reinterpret_cast<float*>(a + kImg)[64 * O_CQ + i] = p.q_scale * s.rn[64 + i] * inverse_pow2(fa);
#pragma unroll 1
      for (int j0 = 0; j0 < 64; j0 += 16) {
        float x[16] = {};
        if (j0 < last) block(j0, x);
        uint32_t w[8], wl[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) split2(make_float2(x[2 * k] * fa, x[2 * k + 1] * fa), &w[k], &wl[k]);
        store_pair(a, i, j0, w);
        store_pair(a + 8192, i, j0, wl);
      }
    }
    if (lower) {
      // T = (I + L)^-1, in place of L. First its diagonal blocks of 16, a column a
      // thread: t_i = [i = col] - sum_{l < i} L_il t_l.
      const int c16 = i & 15;
      float* L = s.m[hd] + (i & 48) * (kLStride + 1);
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
    meet();
    // Then twice the size at a time: [T11 0; L21 .] -> T21 = -T22 (L21 T11).
    {
      const int o = (q >> 6) * 32, r = (q & 63) >> 2, cc = (q & 3) * 4;
      float* m = s.m[hd] + o * (kLStride + 1);
      float* x = s.x[hd] + (q >> 6) * 16 * kXStride;
      float4 v[1] = {};
      mac4(v, m + (16 + r) * kLStride, kLStride, m + cc, kLStride, 0, 16);
      *reinterpret_cast<float4*>(x + r * kXStride + cc) = v[0];
      meet();
      v[0] = make_float4(0.f, 0.f, 0.f, 0.f);
      mac4(v, m + (16 + r) * kLStride + 16, kLStride, x + cc, kXStride, 0, 16);
      *reinterpret_cast<float4*>(m + (16 + r) * kLStride + cc) = minus(v[0]);
      meet();
    }
    {
      const int r = (q >> 3) * 2, cc = (q & 7) * 4;
      float *m = s.m[hd], *x = s.x[hd];
      float4 v[2] = {};
      mac4(v, m + (32 + r) * kLStride, kLStride, m + cc, kLStride, cc & 16, 32);  // T11 is 0 above its diagonal
      *reinterpret_cast<float4*>(x + r * kXStride + cc) = v[0];
      *reinterpret_cast<float4*>(x + (r + 1) * kXStride + cc) = v[1];
      meet();
      v[0] = v[1] = make_float4(0.f, 0.f, 0.f, 0.f);
      mac4(v, m + (32 + r) * kLStride + 32, kLStride, x + cc, kXStride, 0, (r & 16) + 16);  // and so is T22
      *reinterpret_cast<float4*>(m + (32 + r) * kLStride + cc) = minus(v[0]);
      *reinterpret_cast<float4*>(m + (33 + r) * kLStride + cc) = minus(v[1]);
      meet();
    }
#pragma unroll
    for (int u = q; u < 256; u += 128) {
      const int r = u >> 2, j = (u & 3) * 16;
      uint32_t w[8] = {}, wl[8] = {};
      if (j <= r) {  // T is 0 above its diagonal (in m only the diagonal blocks are)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 y = *reinterpret_cast<const float4*>(s.m[hd] + r * kLStride + j + 4 * k);
          split2(make_float2(y.x * kScaleT, y.y * kScaleT), &w[2 * k], &wl[2 * k]);
          split2(make_float2(y.z * kScaleT, y.w * kScaleT), &w[2 * k + 1], &wl[2 * k + 1]);
        }
      }
      store_pair(img, r, j, w);
      store_pair(img + 8192, r, j, wl);
    }
    meet();  // before the next head's gates and L
  }
  if (warp == kStoreWarp && lane == 0) bulk_wait_all();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 64);
  // This kernel needs nothing of the recurrent one, which it overlaps, but ends after it:
  // what comes next in the stream waits for both.
  griddep_wait();
}

// ------------------------------------------------------------------ the chunks of a sequence

// Warps: 0 and 2 load, 1 issues MMAs, 3 looks each chunk's v over; 4 to 11 keep the state's rows (a
// thread is a row of S^T and half of its columns, or of the chunk's tokens); 12 to 19
// write the outputs, half of the tokens each four.
// The loops over columns and tokens are rolled, 16 at a time: one warp a scheduler in
// code that runs straight through waits for its instructions (unrolled, a chunk took 4
// times as long).
constexpr int kChainThreads = 640;

// TMEM columns
constexpr uint32_t kS = 0, kShi = 128, kSlo = 192, kPU = 256, kRhi = 320, kRlo = 352, kQS = 384, kAU = 448;
// U for the outputs, in the upper halves of S lo and S hi: what reads those is done
// when U is known
constexpr uint32_t kUhi = kSlo + 32, kUlo = kShi + 32;

template <int D>
struct alignas(1024) ChainIn {
  unsigned char k[64 * D * 2];  // f16 image
  unsigned char thi[8192], tlo[8192];
  float scal[S_COUNT][64];
  __nv_bfloat16 v[64][D];
};
// When the chunk's products are done, the outputs are staged over the images
// ([token][D] f32).
template <int D>
struct alignas(1024) OutIn {
  unsigned char q[64 * D * 2];
  unsigned char ahi[8192], alo[8192];
  float scal[O_COUNT][64];
};

// Chunks of inputs in shared memory: what the chain needs three deep (a chunk's scales
// are worked out a chunk ahead, and a load takes most of a chunk's time), what the
// outputs need two deep.
constexpr int kIn = 3;
__device__ __forceinline__ int in_stage(int n) { return n % kIn; }
__device__ __forceinline__ uint32_t in_phase(int n) { return (n / kIn) & 1; }

template <int D>
struct ChainSmem {
  ChainIn<D> in[kIn];
  OutIn<D> oin[2];
  float part[2][128];   // of a row's squares, by halves of its columns
  float inv_s[2][128], inv_u[2][128];
  int first_bad[2][128];
  // Of a chunk, for its scales: with v a row's largest |v| (v_max, as bf16), bounds of R and
  // U as [0] v + [1] |S0|, of the state after it as [2] |S0| + [3] v; and whether all its v,
  // k and gates are finite.
  uint16_t v_max[kIn][D];
  float4 scale[kIn];
  int finite_in[kIn];
  uint64_t full[kIn], empty[kIn], v_ready[kIn], ofull[2], oempty[2], s_ready[2], s_done[2];
  uint64_t p_done, r_ready, u_done, u_ready, o_done, o_free, row_ready, state_in, state_read;
  uint32_t tmem;
};

// silu(z) before a rounding to bf16: the fast exponential and division (a few 2^-22)
// are far below it.
__device__ __forceinline__ float2 gate(float2 z) {
  const float2 t = __fmul2_rn(z, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return __fmul2_rn(z, r);
}

// A state passes through shared memory on its way in (where the outputs' inputs come
// later) and out (where the chain's were): a thread's row at a time from global memory, the
// two took 7 us a CTA. Rows 16 bytes further apart than they are long: no bank conflicts.
template <int D, bool BF16>
constexpr int state_row() { return D * (BF16 ? 2 : 4) + 16; }

// 16 columns of a row of a state in shared memory.
template <bool BF16>
__device__ __forceinline__ void state16(const unsigned char* row, int col, float (&x)[16]) {
  if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + 2 * col + 16 * j);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) x[8 * j + 2 * k] = bf16_lo(w[k]), x[8 * j + 2 * k + 1] = bf16_hi(w[k]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(row + 4 * col + 16 * j);
      x[4 * j] = v.x, x[4 * j + 1] = v.y, x[4 * j + 2] = v.z, x[4 * j + 3] = v.w;
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kChainThreads, 1) delta_kernel(const ChunkParams c) {
  const DeltaParams& p = c.p;
  extern __shared__ unsigned char raw[];
  ChainSmem<D>& s = *reinterpret_cast<ChainSmem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  const int h = blockIdx.x, kh = h / p.group;
  const int sq = p.order ? __ldcg(p.order + blockIdx.y) : blockIdx.y;
  // four loads: of one of 16 bytes the parts had no uniform registers, and the spills took 3%
  const int* plan = reinterpret_cast<const int*>(p.plan + sq);
  const int b = __ldcg(plan), e = __ldcg(plan + 1), in = __ldcg(plan + 2), out = __ldcg(plan + 3);
  if (e <= b) return;
  const int chunks = (e - b + kChunk - 1) / kChunk, place0 = chunk_first_place(sq, b);
  if (tid == 0) {
    for (int i = 0; i < kIn; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 2);  // the MMAs' commit, and the warp that looks v over
      mbar_init(&s.v_ready[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.ofull[i], 1);
      mbar_init(&s.oempty[i], 9);  // the MMAs' commit, and the output warps
      mbar_init(&s.s_ready[i], 4);
      mbar_init(&s.s_done[i], 1);
    }
    mbar_init(&s.p_done, 1);
    mbar_init(&s.r_ready, 8);
    mbar_init(&s.u_done, 1);
    mbar_init(&s.u_ready, 8);
    mbar_init(&s.o_done, 1);
    mbar_init(&s.o_free, 8);
    mbar_init(&s.row_ready, 4);
    mbar_init(&s.state_in, 1);
    mbar_init(&s.state_read, 8);
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc(&s.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  bool ok = true;
  constexpr int kRow = state_row<D, BF16>(), kRowData = kRow - 16;
  static_assert(D * kRow <= sizeof(s.oin) && D * kRow <= sizeof(s.in), "a state passes through these");

  if (warp == 0) {
    int n = 0;
    for (; n < chunks; ++n) {
      const int t0 = b + n * kChunk, toks = min(kChunk, e - t0), st = in_stage(n);
      const size_t place = place0 + n;
      const unsigned char* kq = c.kq + (place * p.Hk + kh) * kq_bytes<D>();
      const unsigned char* img = c.head + (place * p.Hv + h) * kHeadBytes;
      ChainIn<D>& g = s.in[st];
      ok = ok && mbar_wait(&s.empty[st], in_phase(n) ^ 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&s.full[st], kq_bytes<D>() / 2 + kChainBytes + toks * D * 2);
        bulk_load(g.thi, img, kChainBytes, &s.full[st]);
      }
      __syncwarp();
      for (int t = lane; t < toks; t += 32)
        bulk_load(g.v[t], p.qkv + (long long)(t0 + t) * p.ldqkv + 2 * p.Hk * D + h * D, D * 2, &s.full[st]);
      if (lane == 0) bulk_load(g.k, kq, kq_bytes<D>() / 2, &s.full[st]);
    }
    // no copy is in flight when the CTA leaves
    for (int m = max(0, n - kIn); m < n; ++m) ok = mbar_wait(&s.full[in_stage(m)], in_phase(m)) && ok;
  } else if (warp == 2) {
    if (in > 0) {
      if (lane == 0) mbar_arrive_expect_tx(&s.state_in, D * kRowData);
      __syncwarp();
      const unsigned char* src = static_cast<const unsigned char*>(p.state) + ((size_t)in * p.Hv + h) * D * kRowData;
      for (int r = lane; r < D; r += 32)
        bulk_load(reinterpret_cast<unsigned char*>(s.oin) + r * kRow, src + r * kRowData, kRowData, &s.state_in);
      ok = mbar_wait(&s.state_read, 0);
      ok = __all_sync(0xffffffffu, ok);
    }
    // what the outputs need, with a wait of its own: the outputs may lag behind the chain
    int n = 0;
    for (; n < chunks; ++n) {
      const int st = n & 1;
      ok = ok && mbar_wait(&s.oempty[st], ((n >> 1) & 1) ^ 1);
      if (!ok) break;
      const size_t place = place0 + n;
      if (elect_one()) {
        OutIn<D>& y = s.oin[st];
        mbar_arrive_expect_tx(&s.ofull[st], kq_bytes<D>() / 2 + kOutBytes);
        bulk_load(y.q, c.kq + (place * p.Hk + kh) * kq_bytes<D>() + kq_bytes<D>() / 2, kq_bytes<D>() / 2, &s.ofull[st]);
        bulk_load(y.ahi, c.head + (place * p.Hv + h) * kHeadBytes + kChainBytes, kOutBytes, &s.ofull[st]);
      }
      __syncwarp();
    }
    for (int m = max(0, n - 2); m < n; ++m) ok = mbar_wait(&s.ofull[m & 1], (m >> 1) & 1) && ok;
    if (!ok && in > 0) mbar_wait(&s.state_in, 0);
  } else if (warp == 1) {
    // the whole warp waits, one lane issues
    constexpr uint32_t idesc = idesc_f16(128, 64, false), idesc_s = idesc_f16(128, 64, true);
    // T and the causal products are zero above their diagonals: 16 of their columns meet
    // the rows from there down. In a descriptor, 16 rows and 16 columns on.
    constexpr int kDown = 128 + 2;
    for (int n = 0; n < chunks && ok; ++n) {
      const int st = n & 1;
      const uint32_t ph = n & 1;
      ChainIn<D>& g = s.in[in_stage(n)];
      OutIn<D>& y = s.oin[st];
      const uint64_t kd = sdesc_k_sw128(smem_u32(g.k)), qd = sdesc_k_sw128(smem_u32(y.q));
      if (!(ok = mbar_wait(&s.full[in_stage(n)], in_phase(n)))) break;
      // P = S k, in halves of dk as they are ready
      if (!(ok = mbar_wait(&s.s_ready[0], ph))) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint64_t bd = kd + (j >> 2) * 512 + 2 * (j & 3);
          mma_f16_ts(tmem + kPU, tmem + kShi + 8 * j, bd, idesc, j > 0);
          mma_f16_ts(tmem + kPU, tmem + kSlo + 8 * j, bd, idesc, true);
        }
      }
      __syncwarp();
      if (!(ok = mbar_wait(&s.s_ready[1], ph))) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int j = D / 32; j < D / 16; ++j) {
          const uint64_t bd = kd + (j >> 2) * 512 + 2 * (j & 3);
          mma_f16_ts(tmem + kPU, tmem + kShi + 8 * j, bd, idesc, true);
          mma_f16_ts(tmem + kPU, tmem + kSlo + 8 * j, bd, idesc, true);
        }
        mma_commit(&s.p_done);
      }
      __syncwarp();
      // the state's part of the outputs, under the chain
      if (!(ok = mbar_wait(&s.ofull[st], (n >> 1) & 1))) break;
      if (!(ok = mbar_wait(&s.o_free, ph ^ 1))) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint64_t bd = qd + (j >> 2) * 512 + 2 * (j & 3);
          mma_f16_ts(tmem + kQS, tmem + kShi + 8 * j, bd, idesc, j > 0);
          mma_f16_ts(tmem + kQS, tmem + kSlo + 8 * j, bd, idesc, true);
        }
      }
      __syncwarp();
      // U = R T^T
      if (!(ok = mbar_wait(&s.r_ready, ph))) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t th = sdesc_k_sw128(smem_u32(g.thi)), tl = sdesc_k_sw128(smem_u32(g.tlo));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t id = idesc_f16(128, 64 - 16 * j, false), d = tmem + kPU + 16 * j;
          mma_f16_ts(d, tmem + kRhi + 8 * j, th + kDown * j, id, j > 0);
          mma_f16_ts(d, tmem + kRhi + 8 * j, tl + kDown * j, id, true);
          mma_f16_ts(d, tmem + kRlo + 8 * j, th + kDown * j, id, true);
        }
        mma_commit(&s.u_done);
      }
      __syncwarp();
      // S += U' k, 64 columns of dk at a time (U' hi, lo stand where R's were)
      if (!(ok = mbar_wait(&s.u_ready, ph))) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t km = sdesc_mn_sw128(smem_u32(g.k), 8192);
#pragma unroll
        for (int a = 0; a < D / 64; ++a) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t bd = km + a * 512 + j * 128;
            mma_f16_ts(tmem + kS + a * 64, tmem + kRhi + 8 * j, bd, idesc_s, true);
            mma_f16_ts(tmem + kS + a * 64, tmem + kRlo + 8 * j, bd, idesc_s, true);
          }
          mma_commit(&s.s_done[a]);
        }
        if (D == 64) mma_commit(&s.s_done[1]);
        mma_commit(&s.empty[in_stage(n)]);
        const uint64_t ah = sdesc_k_sw128(smem_u32(y.ahi)), al = sdesc_k_sw128(smem_u32(y.alo));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t id = idesc_f16(128, 64 - 16 * j, false), d = tmem + kAU + 16 * j;
          mma_f16_ts(d, tmem + kUhi + 8 * j, ah + kDown * j, id, j > 0);
          mma_f16_ts(d, tmem + kUlo + 8 * j, ah + kDown * j, id, true);
          mma_f16_ts(d, tmem + kUhi + 8 * j, al + kDown * j, id, true);
        }
        mma_commit(&s.o_done);
        mma_commit(&s.oempty[st]);
      }
      __syncwarp();
    }
    // no MMA is in flight when the TMEM is freed
    if (ok) ok = mbar_wait(&s.o_done, (chunks - 1) & 1);
  } else if (warp == 3) {
    // each row's largest |v| of the chunk, from the bits (a NaN or an infinity is larger than any)
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    for (int n = 0; n < chunks; ++n) {
      const int st = in_stage(n), toks = min(kChunk, e - (b + n * kChunk));
      if (ok) ok = mbar_wait(&s.full[st], in_phase(n));
      // eight rows of S^T a lane (columns of v), their largest of every kRows-th token
      uint4 m = make_uint4(0, 0, 0, 0);
      const auto look = [&](int t) {
        const uint4 v = *reinterpret_cast<const uint4*>(&s.in[st].v[t][lane % kLanes * 8]);
        m.x = __vmaxu2(m.x, v.x & 0x7fff7fffu), m.y = __vmaxu2(m.y, v.y & 0x7fff7fffu);
        m.z = __vmaxu2(m.z, v.z & 0x7fff7fffu), m.w = __vmaxu2(m.w, v.w & 0x7fff7fffu);
      };
      if (toks == kChunk) {
#pragma unroll 8
        for (int t = 0; t < kChunk; t += kRows) look(t + lane / kLanes);
      } else {
        for (int t = lane / kLanes; t < toks; t += kRows) look(t);
      }
#pragma unroll
      for (int o = 16; o >= kLanes; o >>= 1) {
        m.x = __vmaxu2(m.x, __shfl_xor_sync(0xffffffffu, m.x, o)), m.y = __vmaxu2(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
        m.z = __vmaxu2(m.z, __shfl_xor_sync(0xffffffffu, m.z, o)), m.w = __vmaxu2(m.w, __shfl_xor_sync(0xffffffffu, m.w, o));
      }
      if (lane < kLanes) *reinterpret_cast<uint4*>(&s.v_max[st][lane * 8]) = m;
      const uint32_t two = __vmaxu2(__vmaxu2(m.x, m.y), __vmaxu2(m.z, m.w));
      const uint32_t all = __reduce_max_sync(0xffffffffu, max(two & 0xffffu, two >> 16));
      __syncwarp();  // v_max, before the arrival
      if (lane == 0) {
        const float4 end = *reinterpret_cast<const float4*>(s.in[st].scal[S_END]);
        const float2 rest = *reinterpret_cast<const float2*>(&s.in[st].scal[S_END][4]);
        s.scale[st] = make_float4(end.z * (1.f + end.w), rest.y, end.x, rest.x);
        s.finite_in[st] = __float_as_int(end.y) == kChunk && all < 0x7f80;
        mbar_arrive(&s.v_ready[st]);
        mbar_arrive(&s.empty[st]);
      }
      __syncwarp();
    }
  } else if (warp >= 4 && warp < 12) {
    // ---- the state's rows
    const int row = tid & 127, half = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int col0 = half * (D / 2), tok0 = half * 32;
    const bool real = row < D;
    // The lanes past D = 64 rows do as the first 64 do, from a zero state; nobody
    // reads them.
    const int vrow = row & (D - 1);
    // bound: of the row's 2-norm at the chunk's start, which fs is the scale of
    float bound, fs;
    bool dead;  // the row holds a value that is not finite
    {
      // this thread's half of the row
      float x[D / 32][16] = {};
      float zero = 0.f, mx = 0.f;
      if (in > 0) ok = mbar_wait(&s.state_in, 0);
      if (real && in > 0) {
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          state16<BF16>(reinterpret_cast<const unsigned char*>(s.oin) + row * kRow, col0 + 16 * k, x[k]);
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
#pragma unroll
          for (int j = 0; j < 16; ++j) mx = fmaxf(mx, fabsf(x[k][j])), zero += x[k][j] * 0.f;
      }
      __syncwarp();
      if (in > 0 && lane == 0) mbar_arrive(&s.state_read);
      s.part[half][row] = zero == 0.f ? mx : __int_as_float(0x7fffffff);
      asm volatile("bar.sync 2, 256;" ::: "memory");
      const float a = s.part[0][row], o = s.part[1][row];
      dead = !(finite(a) && finite(o));
      bound = dead ? 0.f : fminf(12.f * fmaxf(a, o), kLargest);  // at least the 2-norm of 128 values
      fs = row_scale(bound);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[k][j] = dead ? 0.f : x[k][j] * fs;
        tmem_st16f(tmem + kS + col0 + 16 * k + lanes, x[k]);
      }
      tmem_wait_st();
    }
    // A chunk's scales, worked out while the chunk before waits for its U: first_bad,
    // the first token not finite; fu, of U; fs_next, of the state after the chunk;
    // shrink, what takes S from one to the other.
    // added, the bound's part from v.
    int first_bad = 0;
    float fu = 1.f, fs_next = 1.f, shrink = 0.f, added = 0.f;
    const auto scales = [&](int n) {
      const int st = in_stage(n), toks = min(kChunk, e - (b + n * kChunk));
      ChainIn<D>& g = s.in[st];
      if (ok) ok = mbar_wait(&s.v_ready[st], in_phase(n));  // after full[st]
      float4 k = s.scale[st];
      const float most = __uint_as_float((uint32_t)s.v_max[st][vrow] << 16);
      k.x *= most, k.w *= most;
      first_bad = kChunk;
      if (!s.finite_in[st]) {
        // up to the first token of this row whose v, k or gates are not finite
        const float4 end = *reinterpret_cast<const float4*>(g.scal[S_END]);
        float mv = 0.f;
        first_bad = __float_as_int(end.y);
        for (int i = 0; i < min(toks, first_bad); ++i) {
          const float a = fabsf(bf16_to_f(g.v[i][vrow]));
          if (!finite(a))
            first_bad = i;
          else
            mv = fmaxf(mv, a);
        }
        k = first_bad < kChunk ? make_float4((1.f + kChunk) * mv, 1.f, 0.f, 0.f)
                               : make_float4(end.z * (mv + mv * end.w), g.scal[S_END][5], end.x, g.scal[S_END][4] * mv);
      }
      if (dead) first_bad = 0, k.z = k.w = 0.f;
      fu = row_scale(fmaf(k.y, bound, k.x));
      added = k.w;
      bound = fminf(fmaf(k.z, bound, added) * 1.01f, kLargest);
      fs_next = row_scale(bound);
      shrink = k.z * fminf(fs_next * inverse_pow2(fs), 0x1p126f);
    };
    scales(0);
    for (int n = 0; n < chunks; ++n) {
      const int st = n & 1, toks = min(kChunk, e - (b + n * kChunk));
      const uint32_t ph = n & 1;
      ChainIn<D>& g = s.in[in_stage(n)];
      const float inv_s = inverse_pow2(fs), p_scale = fminf(fu * inv_s, 0x1p127f);
      const float u_scale = fminf(fs_next * inverse_pow2(fu), 0x1p126f);
      const int until = min(first_bad, toks);  // R is zero from there on
      const bool bad = first_bad < kChunk;
      if (half == 0) {
        s.inv_s[st][row] = inv_s;
        s.inv_u[st][row] = inverse_pow2(fu);
        s.first_bad[st][row] = first_bad;
      }
      if (n > 0) {
        if (ok) ok = mbar_wait(&s.s_done[half], ph ^ 1);
        if (half == 1 && ok) ok = mbar_wait(&s.o_done, ph ^ 1);  // U stood in the upper halves
        tc_fence_after();
      }
      // S hi, lo for this chunk's products, and S shrunk for what is added to it
      float2 ss2 = make_float2(0.f, 0.f);
      const bool measure = (n & 7) == 7;
      const float2 shrink2 = make_float2(shrink, shrink);
#pragma unroll 1
      for (int col = col0; col < col0 + D / 2; col += 16) {
        float x[16];
        uint32_t hi[8], lo[8];
        tmem_ld16(tmem + kS + col + lanes, x);
        if (dead) {
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = 0.f;
        }
        if (measure) {
#pragma unroll
          for (int j = 0; j < 16; j += 2) ss2 = __ffma2_rn(make_float2(x[j], x[j + 1]), make_float2(x[j], x[j + 1]), ss2);
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 y = make_float2(x[j], x[j + 1]);
          split2(y, &hi[j / 2], &lo[j / 2]);
          const float2 z = __fmul2_rn(y, shrink2);
          x[j] = z.x, x[j + 1] = z.y;
        }
        tmem_st8(tmem + kShi + col / 2 + lanes, hi);
        tmem_st8(tmem + kSlo + col / 2 + lanes, lo);
        tmem_st16f(tmem + kS + col + lanes, x);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.s_ready[half]);
      // R, with this row's v read ahead
      uint32_t v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        v[j] = __bfloat16_as_ushort(g.v[tok0 + 2 * j][vrow]) | ((uint32_t)__bfloat16_as_ushort(g.v[tok0 + 2 * j + 1][vrow]) << 16);
      const float2 p2 = make_float2(-p_scale, -p_scale);
      const uint16_t fu_bf16 = (uint16_t)(__float_as_uint(fu) >> 16);  // a power of two
      if (ok) ok = mbar_wait(&s.p_done, ph);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = tok0 + 16 * k;
        float x[16];
        uint32_t hi[8], lo[8];
        tmem_ld16(tmem + kPU + i + lanes, x);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float4 rc = *reinterpret_cast<const float4*>(&g.scal[S_R][2 * (i + j)]);
          const float2 q = __fmul2_rn(__fmul2_rn(make_float2(x[j], x[j + 1]), make_float2(rc.z, rc.w)), p2);
          const float2 r = __fmul2_rn(add_scaled(v[8 * k + j / 2], fu_bf16, q), make_float2(rc.x, rc.y));
          x[j] = r.x, x[j + 1] = r.y;
        }
        if (until < kChunk) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (i + j >= until) x[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) split2(make_float2(x[j], x[j + 1]), &hi[j / 2], &lo[j / 2]);
        tmem_st8(tmem + kRhi + i / 2 + lanes, hi);
        tmem_st8(tmem + kRlo + i / 2 + lanes, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.r_ready);
      // the next chunk's scales, while U is worked out
      const int bad_from = first_bad;
      if (measure) {
        // the norm of S before this chunk, its halves put together, tightens the bound after it
        s.part[half][row] = ss2.x + ss2.y;
        asm volatile("bar.sync 2, 256;" ::: "memory");
        const float norm = sqrtf(s.part[0][row] + s.part[1][row]) * inv_s;
        bound = fminf(bound, fmaf(shrink * fs, norm * inverse_pow2(fs_next), added) * 1.01f);
      }
      fs = fs_next;
      if (bad) dead = true;  // from the next chunk on
      if (n + 1 < chunks) scales(n + 1);
      // U for the outputs, and e^(G_C-G) U at the state's scale
      const float2 us2 = make_float2(u_scale, u_scale), t2 = make_float2(1.0f / kScaleT, 1.0f / kScaleT);
      if (ok) ok = mbar_wait(&s.u_done, ph);
      tc_fence_after();
#pragma unroll 2
      for (int i = tok0; i < tok0 + 32; i += 16) {
        float u[16];
        uint32_t hi[8], lo[8], ohi[8], olo[8];
        tmem_ld16(tmem + kPU + i + lanes, u);
        if (bad) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (i + j >= bad_from) u[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float4 c4 = *reinterpret_cast<const float4*>(&g.scal[S_CU][i + (j & ~3)]);
          const float2 cu = j & 2 ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
          const float2 y = __fmul2_rn(make_float2(u[j], u[j + 1]), t2);
          split2(y, &ohi[j / 2], &olo[j / 2]);
          float2 w = __fmul2_rn(__fmul2_rn(y, cu), us2);
          if (bad) w = make_float2(0.f, 0.f);
          split2(w, &hi[j / 2], &lo[j / 2]);
        }
        tmem_st8(tmem + kRhi + i / 2 + lanes, hi);
        tmem_st8(tmem + kRlo + i / 2 + lanes, lo);
        tmem_st8(tmem + kUhi + i / 2 + lanes, ohi);
        tmem_st8(tmem + kUlo + i / 2 + lanes, olo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      // row_ready goes with u_ready, not before: this chunk's U waited for the
      // outputs of the chunk before (o_free), so row_ready never runs two phases
      // ahead of the output warps
      if (lane == 0) {
        mbar_arrive(&s.u_ready);
        if (half == 0) mbar_arrive(&s.row_ready);
      }
    }
    // the state after the last chunk, through the room of the chain's inputs: every MMA that
    // reads them is done
    if (ok) ok = mbar_wait(&s.s_done[1], (chunks - 1) & 1);
    tc_fence_after();
    const float nan = __int_as_float(0x7fffffff), inv = inverse_pow2(fs);
    constexpr int kHalf = kRowData / 2;  // bytes of this thread's half of the row
    unsigned char* mine = reinterpret_cast<unsigned char*>(s.in) + row * kRow + half * kHalf;
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 16) {
      float x[16];
      tmem_ld16(tmem + kS + col0 + c + lanes, x);
      if (!real || !ok) continue;
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = dead ? nan : x[j] * inv;
      if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<uint4*>(mine + 2 * c + 16 * j) =
              make_uint4(pack_bf16x2(x[8 * j], x[8 * j + 1]), pack_bf16x2(x[8 * j + 2], x[8 * j + 3]),
                         pack_bf16x2(x[8 * j + 4], x[8 * j + 5]), pack_bf16x2(x[8 * j + 6], x[8 * j + 7]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(mine + 4 * c + 16 * j) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      }
    }
    if (real && ok) {
      fence_proxy_async_smem();
      bulk_store(static_cast<unsigned char*>(p.state) + (((size_t)out * p.Hv + h) * D + row) * kRowData + half * kHalf, mine, kHalf);
      bulk_commit();
      bulk_wait_all();
    }
  } else if (warp >= 12) {
    // ---- the outputs
    const int row = tid & 127, w = warp - 12, half = w >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // On the way out eight lanes take a row, four columns in every 32 each; a warp
    // the rows 8 w .. 8 w + 7, four at a time.
    constexpr int E = D / 32;
    const int sub = lane >> 3, l8 = (lane & 7) * 4;
    for (int n = 0; n < chunks; ++n) {
      const int st = n & 1, t0 = b + n * kChunk, toks = min(kChunk, e - t0);
      const uint32_t ph = n & 1;
      OutIn<D>& y = s.oin[st];
      float* o32 = reinterpret_cast<float*>(y.q);
      // this warp's rows of z, in flight while the chunk is finished
      uint2 z[2][E];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 8 * w + 4 * i + sub;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          z[i][k] = make_uint2(0, 0);
          if (p.z && t < toks)
            z[i][k] = __ldg(reinterpret_cast<const uint2*>(p.z + (long long)(t0 + t) * p.ldz + h * D + 32 * k + l8));
        }
      }
      if (ok) ok = mbar_wait(&s.row_ready, ph);
      if (ok) ok = mbar_wait(&s.ofull[st], (n >> 1) & 1);
      const float2 is2 = make_float2(s.inv_s[st][row], s.inv_s[st][row]), iu2 = make_float2(s.inv_u[st][row], s.inv_u[st][row]);
      const int first_bad = s.first_bad[st][row];
      if (ok) ok = mbar_wait(&s.o_done, ph);
      tc_fence_after();
#pragma unroll 1
      for (int i = 32 * half; i < 32 * half + 32; i += 16) {
        float x[16], u[16];
        tmem_ld16(tmem + kQS + i + lanes, x);
        tmem_ld16(tmem + kAU + i + lanes, u);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 cg = *reinterpret_cast<const float4*>(&y.scal[O_CQG][i + j]);
          const float4 cq = *reinterpret_cast<const float4*>(&y.scal[O_CQ][i + j]);
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float2 a = __fmul2_rn(k ? make_float2(cg.z, cg.w) : make_float2(cg.x, cg.y), is2);
            const float2 w = __fmul2_rn(k ? make_float2(cq.z, cq.w) : make_float2(cq.x, cq.y), iu2);
            const float2 o = __ffma2_rn(make_float2(x[j + k], x[j + k + 1]), a, __fmul2_rn(make_float2(u[j + k], u[j + k + 1]), w));
            u[j + k] = o.x, u[j + k + 1] = o.y;
          }
        }
        if (first_bad < i + 16) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (i + j >= first_bad) u[j] = __int_as_float(0x7fffffff);
        }
        if (row < D) {
#pragma unroll
          for (int j = 0; j < 16; ++j) o32[(i + j) * D + row] = u[j];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_free);
      asm volatile("bar.sync %0, 128;" ::"r"(3 + half) : "memory");  // this half's rows are staged
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 8 * w + 4 * i + sub;
        float4 o[E];
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] = *reinterpret_cast<const float4*>(o32 + t * D + 32 * k + l8);
        if (p.z) {
          float2 ss = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float2 a = make_float2(o[k].x, o[k].y), b = make_float2(o[k].z, o[k].w);
            ss = __ffma2_rn(a, a, __ffma2_rn(b, b, ss));
          }
          float sum = ss.x + ss.y;
#pragma unroll
          for (int m = 4; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
          const float r = rsqrtf(sum * (1.0f / D) + p.gnorm_eps);
          const float2 r2 = make_float2(r, r);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const uint2 gw = __ldg(reinterpret_cast<const uint2*>(p.gnorm_w + 32 * k + l8));
            const auto out = [&](float2 v, uint32_t g, uint32_t zz) {
              const float2 w = __fmul2_rn(__fmul2_rn(v, r2), make_float2(bf16_lo(g), bf16_hi(g)));
              return __fmul2_rn(w, gate(make_float2(bf16_lo(zz), bf16_hi(zz))));
            };
            const float2 a = out(make_float2(o[k].x, o[k].y), gw.x, z[i][k].x), b = out(make_float2(o[k].z, o[k].w), gw.y, z[i][k].y);
            o[k] = make_float4(a.x, a.y, b.x, b.y);
          }
        }
        if (t < toks) {
          __nv_bfloat16* dst = p.out + (long long)(t0 + t) * p.ldo + h * D + l8;
#pragma unroll
          for (int k = 0; k < E; ++k)
            *reinterpret_cast<uint2*>(dst + 32 * k) = make_uint2(pack_bf16x2(o[k].x, o[k].y), pack_bf16x2(o[k].z, o[k].w));
        }
      }
      fence_proxy_async_smem();  // the next images come by bulk copies
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.oempty[st]);
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
  const dim3 places((unsigned)(chunk_places(c.p.r.tokens, c.p.r.seqs) - 1) * c.p.Hk);  // the last is the pad rows'
  // Each may start while the kernel before it ends.
  const Launch first(places, kPrepThreads, prep, true, s), second(dim3(c.p.Hv, c.p.r.seqs), kChainThreads, chain, true, s);
  e = cudaLaunchKernelEx(&first.cfg, prepare_kernel<D>, c);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&second.cfg, delta_kernel<D, BF16>, c);
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
  c.ahead = 2 * 152;
  c.head = ws + (size_t)chunk_places(p.r.tokens, p.r.seqs) * p.Hk * 2 * kChunk * d * 2;
  if (d == 128) return state_bf16 ? launch<128, true>(c, s) : launch<128, false>(c, s);
  return state_bf16 ? launch<64, true>(c, s) : launch<64, false>(c, s);
}

}  // namespace gdn
