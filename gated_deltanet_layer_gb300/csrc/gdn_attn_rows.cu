// Paged attention (gdn_attn_paged) on tiles of 16 query rows: one new token a request, or
// a few.
//
// o = sum_p w_p v_p / sum_p w_p with w_p = 2^(x_p - m), x_p = scale log2(e) q . k_p and m
// the running maximum, over the keys once. A task's 16 rows are the G query heads of a
// key/value head times the request's tokens, so every key and value is read once for all of
// them. A tile of keys is 16 for each warp; a warp has its own maximum, sums and
// outputs, its own ring of key and value rows in shared memory, and waits for no other until the
// task's end, where the warps' outputs are added up. Products by mma.sync (16 x 8 x 16),
// which leaves scores and outputs in registers; it has the time: bound by the bandwidth
// of the keys and values.
#include <climits>

#include "gdn_attn.cuh"
#include "gdn_host.h"
#include "gdn_prefill.cuh"
#include "gdn_tc_ptx.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kM = kAttnRowsM;
constexpr int kMergeCols = 32, kMergeStride = 36;  // columns merged at a time; floats of a row, against bank conflicts

template <int D>
struct Rows {
  static constexpr int kW = D == 256 ? 4 : 8;  // warps
  static constexpr int kKT = 16 * kW;          // keys of a tile
  static constexpr int kStages = D == 64 ? 5 : 3;
  static constexpr int kRow = 2 * D;  // bytes of a key row
};

template <int D>
struct RowsSmem {
  using C = Rows<D>;
  unsigned char ring[C::kW][C::kStages][2][16 * C::kRow];  // a warp's stages: keys, values
  unsigned char q[16 * C::kRow];
  float merge[C::kW][kM][kMergeStride];
  float2 ml[C::kW][kM];
  int poison[D];  // the first hidden-from-some key whose value in the column is not finite
  int4 seq[kAttnPlanned + 1];
  long long start[kAttnPlanned + 1];
  PlanScratch<C::kW * 32> scan;
  float2 row_ml[kM];
  int at[4];  // the first unit's request, head, row tile and key tile
  unsigned last;
};

__device__ __forceinline__ void ldmatrix4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte of 16-byte piece c of row r: pieces are permuted within 128 bytes, so that eight rows'
// same pieces are in different banks.
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return r * (2 * D) + ((c ^ (r & 7)) << 4);
}

// One value of a row that is done: divided by the sum, gated.
template <int D>
__device__ __forceinline__ void put2(const AttnParams& p, int row0, int h, int r, int col, float2 v, float l) {
  const uint32_t t = p.group.div(r), g = r - t * p.group.d;
  const long long row = row0 + t;
  const long long c = ((long long)h * p.group.d + g) * D + col;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  v.x *= inv;
  v.y *= inv;
  if (p.gate) {
    const uint32_t z = *reinterpret_cast<const uint32_t*>(p.gate + row * p.ldg + c);
    v.x /= 1.f + __expf(-bf16_lo(z));
    v.y /= 1.f + __expf(-bf16_hi(z));
  }
  *reinterpret_cast<uint32_t*>(p.out + row * p.ldo + c) = pack_bf16x2(v.x, v.y);
}

template <int D>
__global__ void __launch_bounds__(Rows<D>::kW * 32, 1) attn_rows(const AttnParams p) {
  using C = Rows<D>;
  constexpr int W = C::kW, KT = C::kKT, NT = W * 32, ST = C::kStages;
  extern __shared__ unsigned char raw[];
  static_assert(sizeof(RowsSmem<D>) + 128 <= 232448, "227 KB of shared memory a CTA");
  RowsSmem<D>& s = *reinterpret_cast<RowsSmem<D>*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~(uintptr_t)127);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < D; i += NT) s.poison[i] = INT_MAX;
  griddep_wait();
  griddep_launch_dependents();
  const int4* seq = s.seq;
  const long long* start = s.start;
  if (p.seq) {
    seq = p.seq;
    start = p.start;
  } else {
    attn_plan<KT, 0, NT>(p, s.seq, s.start, s.scan, blockIdx.x == 0);
  }
  attn_zero_rows<W>(p, seq, p.Hkv * p.group.d * D);
  const long long units = start[p.seqs];
  const Shares shares(units, (int)min((long long)gridDim.x, (units + 1) / 2));
  if (units == 0 || blockIdx.x >= shares.ctas) return;
  const long long u0 = shares.first(blockIdx.x), u1 = shares.first(blockIdx.x + 1);
  const int steps = (int)(u1 - u0);

  if (warp == 0) Walk<KT, 0>::find(p, seq, start, u0, s.at);
  __syncthreads();

  // The ring's loads: lanes 0 - 15 know the slots of the warp's 16 keys, a step ahead.
  Walk<KT, 0> ahead(p, seq, start);
  ahead.from(s.at, u0);
  const uint32_t ring = smem_u32(s.ring[warp]);
  KeyBlock kb = key_block(p, ahead.s, ahead.j * KT + warp * 16 + (lane & 15), ahead.ctx + ahead.n);
  int issued = 0;
  const auto issue = [&] {
    if (issued < steps) {
      const int slot = key_slot(p, kb, ahead.s);
      const long long col = (long long)ahead.h * D;
      const uint32_t dst = ring + (issued % ST) * (2 * 16 * C::kRow);
      constexpr int kPieces = D / 8, kPer = 32 / kPieces > 0 ? 32 / kPieces : 1;  // rows a warp copies at once
      ++issued;
      if (issued < steps) {
        if (++ahead.j == ahead.nt) ahead.next_task();
        kb = key_block(p, ahead.s, ahead.j * KT + warp * 16 + (lane & 15), ahead.ctx + ahead.n);
      }
#pragma unroll
      for (int r0 = 0; r0 < 16; r0 += kPer) {
        const int r = r0 + lane / kPieces, c = lane % kPieces;
        const int at = __shfl_sync(0xffffffffu, slot, r);
        const long long row = max(at, 0);
        cp_async16_or_zero(dst + piece<D>(r, c), p.k + row * p.ldk + col + c * 8, at >= 0);
        cp_async16_or_zero(dst + 16 * C::kRow + piece<D>(r, c), p.v + row * p.ldv + col + c * 8, at >= 0);
      }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue();

  Walk<KT, 0> w(p, seq, start);
  w.from(s.at, u0);
  float o[D / 8][4], m[2], l[2];
  int last_key[2], first_last = 0;  // last key that the thread's two rows see; the task's first row's
  bool fresh = true;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    if (fresh) {
      fresh = false;
      // the rows' queries; dead rows are zero
      for (int x = tid; x < 16 * D / 8; x += NT) {
        const int r = x / (D / 8), c = x % (D / 8), R = w.i * kM + r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (R < w.n * (int)p.group.d) {
          const uint32_t tok = p.group.div(R), hd = R - tok * p.group.d;
          v = *reinterpret_cast<const uint4*>(p.q + (w.row0 + tok) * p.ldq + ((long long)w.h * p.group.d + hd) * D + c * 8);
        }
        *reinterpret_cast<uint4*>(s.q + piece<D>(r, c)) = v;
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.f;
        last_key[e] = w.ctx + min((int)p.group.div(w.i * kM + g + 8 * e), w.n - 1);
      }
      first_last = w.ctx + p.group.div(w.i * kM);
    }
    issue();
    cp_async_wait_pending(ST - 1);
    __syncwarp();
    const uint32_t ks = ring + (step % ST) * (2 * 16 * C::kRow), vs = ks + 16 * C::kRow, qs = smem_u32(s.q);
    const int key0 = w.j * KT + warp * 16;
    if (key0 < w.ctx + w.n) {
      float x[2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t a[4], b[4];
        ldmatrix4(qs + piece<D>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)), a);
        ldmatrix4(ks + piece<D>((lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1)), b);
        mma16816(x[0], a, b[0], b[1]);
        mma16816(x[1], a, b[2], b[3]);
      }
      const bool edge = key0 + 15 > first_last;  // some row does not see some key
      float top[2] = {m[0], m[1]};
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = x[b][e] * p.scale_log2;
          if (edge && key0 + b * 8 + 2 * t + (e & 1) > last_key[e >> 1]) y = -INFINITY;
          x[b][e] = y;
          top[e >> 1] = fmaxf(top[e >> 1], y);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
        const float f0 = m[0] == -INFINITY ? 0.f : exp2f(m[0] - top[0]), f1 = m[1] == -INFINITY ? 0.f : exp2f(m[1] - top[1]);
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][0] *= f0;
          o[n][1] *= f0;
          o[n][2] *= f1;
          o[n][3] *= f1;
        }
        m[0] = top[0];
        m[1] = top[1];
      }
      const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        x[b][0] = exp2f(x[b][0] - m0);
        x[b][1] = exp2f(x[b][1] - m0);
        x[b][2] = exp2f(x[b][2] - m1);
        x[b][3] = exp2f(x[b][3] - m1);
        l[0] += x[b][0] + x[b][1];
        l[1] += x[b][2] + x[b][3];
      }
      const uint32_t a[4] = {pack_bf16x2(x[0][0], x[0][1]), pack_bf16x2(x[0][2], x[0][3]), pack_bf16x2(x[1][0], x[1][1]),
                             pack_bf16x2(x[1][2], x[1][3])};
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldmatrix4_t(vs + piece<D>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * n + (lane >> 4)), b);
        if (edge && w.n > 1) {
          // 0 x NaN: values that are not finite are taken out where a row does not see their key,
          // and the rows that do see it are told by the column's first such key
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + (e & 1) * 8 + 2 * t;
            int* to = s.poison + n * 16 + (e >> 1) * 8 + g;
            if ((b[e] & 0x7f80u) == 0x7f80u) atomicMin(to, key), b[e] &= 0xffff0000u;
            if ((b[e] & 0x7f800000u) == 0x7f800000u) atomicMin(to, key + 1), b[e] &= 0xffffu;
          }
        }
        mma16816(o[2 * n], a, b[0], b[1]);
        mma16816(o[2 * n + 1], a, b[2], b[3]);
      }
    }
    __syncwarp();
    if (w.j + 1 < w.nt && step + 1 < steps) {
      ++w.j;
      continue;
    }

    // ---- the task's end, or this CTA's: the warps' sums added up
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    if (t == 0) {
      s.ml[warp][g] = make_float2(m[0], l[0]);
      s.ml[warp][g + 8] = make_float2(m[1], l[1]);
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int x = 0; x < W; ++x) top = fmaxf(top, s.ml[x][r].x);
#pragma unroll
      for (int x = 0; x < W; ++x) {
        const float2 ml = s.ml[x][r];
        sum += ml.y * (ml.x == -INFINITY ? 0.f : exp2f(ml.x - top));
      }
      f[e] = m[e] == -INFINITY ? 0.f : exp2f(m[e] - top);
      if (warp == 0 && t == 0) s.row_ml[r] = make_float2(top, sum);
    }
    const long long t0 = w.task, t1 = t0 + w.nt;
    const bool whole = t0 >= u0 && t1 <= u1;
    const int live = min(kM, w.n * (int)p.group.d - w.i * kM);
    const int slot = 2 * blockIdx.x + (t0 >= u0);
    float* part = p.part + (long long)slot * kM * D;
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += kMergeCols) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float* v = o[c0 / 8 + n];
        *reinterpret_cast<float2*>(&s.merge[warp][g][n * 8 + 2 * t]) = make_float2(v[0] * f[0], v[1] * f[0]);
        *reinterpret_cast<float2*>(&s.merge[warp][g + 8][n * 8 + 2 * t]) = make_float2(v[2] * f[1], v[3] * f[1]);
      }
      __syncthreads();
      for (int x = tid; x < kM * kMergeCols / 2; x += NT) {
        const int r = x / (kMergeCols / 2), c = 2 * (x % (kMergeCols / 2));
        if (r < live) {
          float2 v = make_float2(0.f, 0.f);
#pragma unroll
          for (int y = 0; y < W; ++y) {
            const float2 q = *reinterpret_cast<const float2*>(&s.merge[y][r][c]);
            v.x += q.x;
            v.y += q.y;
          }
          const int R = w.i * kM + r, seen = w.ctx + p.group.div(R);
          if (s.poison[c0 + c] <= seen) v.x = NAN;
          if (s.poison[c0 + c + 1] <= seen) v.y = NAN;
          if (whole)
            put2<D>(p, w.row0, w.h, R, c0 + c, v, s.row_ml[r].y);
          else
            *reinterpret_cast<float2*>(part + r * D + c0 + c) = v;
        }
      }
      __syncthreads();
    }
    for (int i = tid; i < D; i += NT) s.poison[i] = INT_MAX;
    if (!whole) {
      if (tid < live) p.part_ml[slot * kM + tid] = s.row_ml[tid];
      const int c0 = shares.owner(t0), c1 = shares.owner(t1 - 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        s.last = atomicAdd(p.done + c0, 1u) == (unsigned)(c1 - c0);
        __threadfence();
      }
      __syncthreads();
      if (s.last) {
        // every part is there: slot 1 of the first CTA, slot 0 of the others (a CTA's part is its
        // second slot where the task begins in it)
        if (tid == 0) p.done[c0] = 0;
        const int parts = c1 - c0 + 1;
        const auto slot_of = [&](int i) { return 2 * (c0 + i) + (i == 0); };
        for (int r = warp; r < live; r += W) {
          float top = -INFINITY, sum = 0.f;
          for (int i = lane; i < parts; i += 32) top = fmaxf(top, __ldcg(&p.part_ml[slot_of(i) * kM + r]).x);
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          for (int i = lane; i < parts; i += 32) {
            const float2 ml = __ldcg(&p.part_ml[slot_of(i) * kM + r]);
            sum += ml.y * (ml.x == -INFINITY ? 0.f : exp2f(ml.x - top));
          }
          sum = warp_sum(sum);
          if (lane == 0) s.row_ml[r] = make_float2(top, sum);
        }
        __syncthreads();
        for (int x = tid; x < live * D / 2; x += NT) {
          const int r = x / (D / 2), c = 2 * (x % (D / 2));
          const float top = s.row_ml[r].x;
          float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
          for (int i = 0; i < parts; ++i) {
            const long long at = slot_of(i) * kM + r;
            const float pm = __ldcg(&p.part_ml[at]).x, e = pm == -INFINITY ? 0.f : exp2f(pm - top);
            const float2 q = __ldcg(reinterpret_cast<const float2*>(p.part + at * D + c));
            v.x = fmaf(q.x, e, v.x);
            v.y = fmaf(q.y, e, v.y);
          }
          put2<D>(p, w.row0, w.h, w.i * kM + r, c, v, s.row_ml[r].y);
        }
      }
    }
    __syncthreads();
    if (step + 1 < steps) w.next_task();
    fresh = true;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(1024) plan_kernel(const AttnParams p) {
  __shared__ PlanScratch<1024> x;
  griddep_wait();
  griddep_launch_dependents();
  attn_plan<Rows<D>::kKT, 0, 1024>(p, p.seq, p.start, x, true);
}

template <int D>
cudaError_t launch(AttnParams p, int grid, cudaStream_t s) {
  const size_t smem = sizeof(RowsSmem<D>) + 128;
  if (p.seqs <= kAttnPlanned) p.seq = nullptr;
  p.tile_m = kM;
  p.tile_g = p.group;
  cudaError_t e = opt_in<attn_rows<D>>(smem);
  if (e != cudaSuccess) return e;
  if (p.seq) {
    const Launch one(dim3(1), 1024, 0, true, s);
    e = cudaLaunchKernelEx(&one.cfg, plan_kernel<D>, p);
    if (e != cudaSuccess) return e;
  }
  const Launch all(dim3(grid), Rows<D>::kW * 32, smem, true, s);
  return cudaLaunchKernelEx(&all.cfg, attn_rows<D>, p);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnParams& p, int d, int grid, cudaStream_t s) {
  return d == 64 ? launch<64>(p, grid, s) : d == 128 ? launch<128>(p, grid, s) : launch<256>(p, grid, s);
}

}  // namespace gdn
