// Paged attention (gdn_attn_paged) on tiles of 16 query rows: one new token a request, or
// a few.
//
// o = sum_p w_p v_p / sum_p w_p with w_p = 2^(x_p - m), x_p = scale log2(e) q . k_p and m
// the running maximum, over the keys once. A task's rows are the G query heads of a
// key/value head times the request's tokens, so every key and value is read once for all of
// them. A tile of keys is 16 for each group of warps (one warp, or two with heads of 256); a
// group has its own maximum, sums and outputs, its own ring of key and value rows in shared
// memory, and waits for no other until the task's end, where the groups' outputs are added up. The rows
// come as boxes of 16 by TMA where blocks are made of 16 slots, else, and past the last key, 16 bytes a
// lane (64 requests over blocks of 24: 107 us for 71 of bandwidth, where boxes take four fifths of it). Products by
// mma.sync (16 x 8 x 16), which leaves scores and outputs in registers; it has the time: the tensor cores are
// busy for a fifth, the issue slots for a quarter.
//
// Bound by the bandwidth of the keys and values. Measured: 64 requests of one token over up to 8192,
// 64 heads of 128 on 8, 926 MB, 165 us (5.6 TB/s, 82% of the measured copy); two over up to 131072, 24 heads of 256 on
// 4, 742 MB, 128 us (5.8 TB/s, 85%; one warp a group of keys 153); one over 100000 of a shard's single key head 23
// (27 with keys and values from memory, of 7.5), of
// which 15 are the plan, the first rows and the joins of 150 parts, in two levels. Rows of several tiles: 20 rows a request and
// key head over up to 6000 read everything twice, 125 us; as a tile of the tensor cores 73.
#include <climits>

#include "gdn_attn.cuh"
#include "gdn_host.h"
#include "gdn_prefill.cuh"
#include "gdn_tc_pair.cuh"

namespace gdn {
namespace {

using namespace tc;

template <int D>
struct Rows {
  static constexpr int kM = 16;                // rows of a task
  // groups of 16 keys of a tile; warps of a group, which share its scores' work twice over and its columns:
  // with heads of 256 four warps alone would not keep up with the rows
  static constexpr int kG = D == 256 ? 4 : 8, kH = D == 256 ? 2 : 1, kW = kG * kH;
  static constexpr int kKT = 16 * kG;          // keys of a tile
  static constexpr int kCols = D / kH;         // a warp's columns of the outputs
  static constexpr int kStages = D == 64 ? 5 : 3;
  static constexpr int kRow = 2 * D;           // bytes of a key row
  // columns merged at a time; floats of a row, against bank conflicts
  static constexpr int kMergeCols = D == 256 ? 16 : 32, kMergeStride = kMergeCols + 4;
};

template <int D>
struct alignas(1024) RowsSmem {
  using C = Rows<D>;
  unsigned char ring[C::kG][C::kStages][2][16 * C::kRow];  // a group's stages: keys, values
  unsigned char q[2][C::kM * C::kRow];  // of a task and the next
  union {
    float merge[C::kW][C::kM][C::kMergeStride];
    float2 parts[16][C::kM];  // the joined parts' maxima and sums
  };
  float2 ml[C::kG][C::kM];
  int poison[D];  // the first hidden-from-some key whose value in the column is not finite
  uint64_t full[C::kG][C::kStages];
  int4 seq[kAttnPlanned + 1];
  long long start[kAttnPlanned + 1];
  PlanScratch<C::kW * 32> scan;
  float2 row_ml[C::kM];
  int at[4];  // the first unit's request, head, row tile and key tile
  unsigned last;
};

// The caches' rows, in boxes of 64 columns and 16 rows; boxes: blocks are made of such.
struct RowMaps {
  CUtensorMap k, v;
  int boxes;
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
// Byte of 16-byte piece c of row r of 16: 64 columns of all rows, then the next; pieces are permuted
// within 128 bytes, so that eight rows' same pieces are in different banks.
__device__ __forceinline__ uint32_t piece(int r, int c) { return (c >> 3) * 2048 + r * 128 + (((c ^ r) & 7) << 4); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two values of a row that is done: divided by the sum, gated.
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
__global__ void __launch_bounds__(Rows<D>::kW * 32, 1) attn_rows(const __grid_constant__ RowMaps maps, const AttnParams p) {
  using C = Rows<D>;
  constexpr int W = C::kW, KT = C::kKT, NT = W * 32, ST = C::kStages, kM = C::kM, kMergeCols = C::kMergeCols;
  extern __shared__ __align__(1024) unsigned char raw[];
  static_assert(sizeof(RowsSmem<D>) <= 232448, "227 KB of shared memory a CTA");
  RowsSmem<D>& s = *reinterpret_cast<RowsSmem<D>*>(raw);
  constexpr int GROUPS = C::kG, HALVES = C::kH;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = warp % GROUPS, hf = warp / GROUPS;
  if (lane == 0 && hf == 0)
    for (int i = 0; i < ST; ++i) mbar_init(&s.full[grp][i], 1);
  // A group's warps wait for one another.
  const auto group_sync = [&] {
    if (HALVES == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * HALVES) : "memory");
  };
  if (tid == 0) {
    if (maps.boxes) prefetch_tensormap(&maps.k), prefetch_tensormap(&maps.v);
  }
  fence_mbar_init();
  for (int i = tid; i < D; i += NT) s.poison[i] = INT_MAX;
  griddep_wait();
  griddep_launch_dependents();
  const int4* seq = s.seq;
  const long long* start = s.start;
  if (p.seq) {
    seq = p.seq;
    start = p.start;
  } else {
    attn_plan<KT, NT>(p, s.seq, s.start, s.scan, blockIdx.x == 0);
  }
  attn_zero_rows<W>(p, seq, p.Hkv * p.group.d * D);
  const long long units = start[p.seqs];
  if (units == 0) return;
  const Shares shares(units, (int)min((long long)gridDim.x, (units + 1) / 2));
  if (blockIdx.x >= shares.ctas) return;
  const long long u0 = shares.first(blockIdx.x), u1 = shares.first(blockIdx.x + 1);
  const int steps = (int)(u1 - u0);

  if (warp == 0) Walk<KT>::find(p, seq, start, u0, s.at);
  __syncthreads();

  // The ring's loads: lanes 0 - 15 know the slots of the warp's 16 keys, a step ahead.
  Walk<KT> ahead(p, seq, start);
  ahead.from(s.at, u0);
  const uint32_t ring = smem_u32(s.ring[grp]);
  const int rows_end = p.num_blocks * (int)p.block.d;
  KeyBlock kb = key_block(p, ahead.s, ahead.j * KT + grp * 16 + (lane & 15), ahead.ctx + ahead.n);
  int issued = 0;
  uint32_t boxed = 0;  // the stages that came as boxes
  // The queries of a task: a share a warp; dead rows are zero. Those of the task after the present one come
  // beside its first step's rows; there is room for no more, so a task of fewer steps than are ahead
  // leaves the one after it to ask for its own.
  int seen = 0, asked = 0, begun = 0;  // tasks: come across by the loads, whose queries are asked for, begun
  const auto queries = [&](const Walk<KT>& x) {
    const uint32_t to = smem_u32(s.q[asked++ & 1]);
    const int rows = x.n * (int)p.group.d;
#pragma unroll 2
    for (int e = tid; e < kM * D / 8; e += NT) {
      const int r = e / (D / 8), c = e % (D / 8), R = x.i * kM + r;
      const bool live = R < rows;
      const uint32_t tok = p.group.div(live ? R : 0), hd = (live ? R : 0) - tok * p.group.d;
      cp_async16_or_zero(to + piece(r, c),
                         p.q + (x.row0 + tok) * p.ldq + ((long long)x.h * p.group.d + hd) * D + c * 8, live);
    }
  };
  bool first = true;  // the next step to be asked for is its task's first here
  bool ok = true;
  const auto issue = [&] {
    if (issued < steps) {
      const int st = issued % ST, slot = key_slot(p, kb, ahead.s), h = ahead.h;
      const bool box = maps.boxes && ahead.j * KT + grp * 16 + 15 < ahead.ctx + ahead.n;
      if (first && seen++ == asked && asked <= begun) queries(ahead);
      first = ahead.j + 1 == ahead.nt;
      ++issued;
      if (issued < steps) {
        if (++ahead.j == ahead.nt) ahead.next_task();
        kb = key_block(p, ahead.s, ahead.j * KT + grp * 16 + (lane & 15), ahead.ctx + ahead.n);
      }
      boxed = box ? boxed | 1u << st : boxed & ~(1u << st);
      if (box) {
        const int row = __shfl_sync(0xffffffffu, slot < 0 ? rows_end : slot, 0);  // past the last row: zeros
        if (lane == 0 && hf == 0) mbar_arrive_expect_tx(&s.full[grp][st], 2 * 16 * C::kRow);
        __syncwarp();
        if (lane < 2 * (D / 64) && hf == 0) {
          const int which = lane / (D / 64), c = lane % (D / 64);
          tma_load_2d_plain(s.ring[grp][st][which] + c * 2048, which ? &maps.v : &maps.k, h * D + c * 64, row, &s.full[grp][st]);
        }
      } else {
        const long long col = (long long)h * D;
        const uint32_t dst = ring + st * (2 * 16 * C::kRow);
        constexpr int kPieces = D / 8, kPer = 32 / kPieces > 0 ? 32 / kPieces : 1;  // rows a warp copies at once
#pragma unroll 2
        for (int r0 = hf * (16 / HALVES); r0 < (hf + 1) * (16 / HALVES); r0 += kPer) {
          const int r = r0 + lane / kPieces, c = lane % kPieces;
          const int at = __shfl_sync(0xffffffffu, slot, r);
          const long long row = max(at, 0);
          cp_async16_or_zero(dst + piece(r, c), p.k + row * p.ldk + col + c * 8, at >= 0);
          cp_async16_or_zero(dst + 16 * C::kRow + piece(r, c), p.v + row * p.ldv + col + c * 8, at >= 0);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue();

  Walk<KT> w(p, seq, start);
  w.from(s.at, u0);
  float o[C::kCols / 8][4], m[2], l[2];
  int last_key[2], first_last = 0;  // last key that the thread's rows see; the task's first row's
  bool fresh = true;
  uint32_t phases = 0;  // of the stages' barriers
  int qbuf = 1;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    const bool starts = fresh;
    if (fresh) {
      fresh = false;
      if (asked == begun) queries(w);
      ++begun;
#pragma unroll
      for (int n = 0; n < C::kCols / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.f;
        last_key[e] = w.ctx + min((int)p.group.div(w.i * kM + g + 8 * e), w.n - 1);
      }
      first_last = w.ctx + p.group.div(w.i * kM);
    }
    issue();
    const int st = step % ST;
    const bool box = boxed >> st & 1;
    if (starts)
      asm volatile("cp.async.wait_all;" ::: "memory");
    else if (!box)
      asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
    if (box) {
      ok = ok && mbar_wait(&s.full[grp][st], phases >> st & 1);
      phases ^= 1u << st;
    }
    if (starts) {
      __syncthreads();  // the other warps' share of the queries
      qbuf ^= 1;
    } else if (!box) {
      group_sync();
    }
    __syncwarp();
    const uint32_t ks = ring + st * (2 * 16 * C::kRow), vs = ks + 16 * C::kRow, qs = smem_u32(s.q[qbuf]);
    const int key0 = w.j * KT + grp * 16;
    if (key0 < w.ctx + w.n) {
      // two sums of a score where the registers allow it: half as many products wait for one another
      constexpr int kSums = D == 256 ? 1 : 2;
      float sums[kSums][2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t a[4], b[4];
        ldmatrix4(ks + piece((lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1)), b);
        ldmatrix4(qs + piece((lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)), a);
        mma16816(sums[k % kSums][0], a, b[0], b[1]);
        mma16816(sums[k % kSums][1], a, b[2], b[3]);
      }
      float x[2][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e >> 2][e & 3] = kSums == 1 ? sums[0][e >> 2][e & 3] : sums[0][e >> 2][e & 3] + sums[kSums - 1][e >> 2][e & 3];
      const bool edge = key0 + 15 > first_last;  // some row does not see some key
      uint32_t a[4];
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
        for (int n = 0; n < C::kCols / 8; ++n) {
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
        float* y = x[b];
        y[0] = ex2(y[0] - m0);
        y[1] = ex2(y[1] - m0);
        y[2] = ex2(y[2] - m1);
        y[3] = ex2(y[3] - m1);
        l[0] += y[0] + y[1];
        l[1] += y[2] + y[3];
        a[2 * b] = pack2(y[0], y[1]);
        a[2 * b + 1] = pack2(y[2], y[3]);
      }
#pragma unroll
      for (int n = 0; n < C::kCols / 16; ++n) {
        uint32_t b[4];
        ldmatrix4_t(vs + hf * (C::kCols / 64 * 2048) + piece((lane & 7) + ((lane >> 3) & 1) * 8, 2 * n + (lane >> 4)), b);
        if (edge && w.n > 1) {
          // 0 x NaN: values that are not finite are taken out where a row does not see their key,
          // and the rows that do see it are told by the column's first such key
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + (e & 1) * 8 + 2 * t;
            int* to = s.poison + hf * C::kCols + n * 16 + (e >> 1) * 8 + g;
            if ((b[e] & 0x7f80u) == 0x7f80u) atomicMin(to, key), b[e] &= 0xffff0000u;
            if ((b[e] & 0x7f800000u) == 0x7f800000u) atomicMin(to, key + 1), b[e] &= 0xffffu;
          }
        }
        mma16816(o[2 * n], a, b[0], b[1]);
        mma16816(o[2 * n + 1], a, b[2], b[3]);
      }
    }
    group_sync();  // the stage is read
    if (w.j + 1 < w.nt && step + 1 < steps) {
      ++w.j;
      continue;
    }

    // ---- the task's end, or this CTA's: the warps' sums added up
    // its last keys are where copies by lanes stand among boxes, and a box may come next in their place
    if (maps.boxes) fence_proxy_async_smem();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (t == 0 && hf == 0) s.ml[grp][g + 8 * e] = make_float2(m[e], l[e]);
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int x = 0; x < GROUPS; ++x) top = fmaxf(top, s.ml[x][r].x);
#pragma unroll
      for (int x = 0; x < GROUPS; ++x) {
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
    for (int c0 = 0; c0 < C::kCols; c0 += kMergeCols) {
#pragma unroll
      for (int n = 0; n < kMergeCols / 8; ++n) {
        const float* v = o[c0 / 8 + n];
        *reinterpret_cast<float2*>(&s.merge[warp][g][n * 8 + 2 * t]) = make_float2(v[0] * f[0], v[1] * f[0]);
        *reinterpret_cast<float2*>(&s.merge[warp][g + 8][n * 8 + 2 * t]) = make_float2(v[2] * f[1], v[3] * f[1]);
      }
      __syncthreads();
      for (int x = tid; x < HALVES * kM * kMergeCols / 2; x += NT) {
        const int h = x / (kM * kMergeCols / 2), r = x / (kMergeCols / 2) % kM, c = 2 * (x % (kMergeCols / 2)), col = h * C::kCols + c0 + c;
        if (r < live) {
          float2 v = make_float2(0.f, 0.f);
#pragma unroll
          for (int y = 0; y < GROUPS; ++y) {
            const float2 q = *reinterpret_cast<const float2*>(&s.merge[h * GROUPS + y][r][c]);
            v.x += q.x;
            v.y += q.y;
          }
          const int R = w.i * kM + r, seen = w.ctx + p.group.div(R);
          if (s.poison[col] <= seen) v.x = NAN;
          if (s.poison[col + 1] <= seen) v.y = NAN;
          if (whole)
            put2<D>(p, w.row0, w.h, R, col, v, s.row_ml[r].y);
          else
            *reinterpret_cast<float2*>(part + r * D + col) = v;
        }
      }
      __syncthreads();
    }
    for (int i = tid; i < D; i += NT) s.poison[i] = INT_MAX;
    if (!whole) {
      if (tid < live) p.part_ml[slot * kM + tid] = s.row_ml[tid];
      // The parts: slot 1 of the first CTA, slot 0 of the others (a CTA's part is its second one
      // where the task begins in it), counted and joined as Join has it.
      const Join join(shares.owner(t0), shares.owner(t1 - 1));
      const int c0 = join.c0;
      const auto slot_of = [&](int i) { return 2 * (c0 + i) + (i == 0); };
      const int mine = join.group(blockIdx.x);
#pragma unroll 1
      for (int level = join.first_level(); level < 2; ++level) {
        const int b = join.begin(level, mine), by = join.step(level), count = join.count(level, mine);
        unsigned* done = p.done + join.word(level, mine, gridDim.x);
        __syncthreads();
        if (tid == 0) s.last = atom_add_acq_rel_u32(done, 1u) == (unsigned)(count - 1);
        __syncthreads();
        if (!s.last) break;
        if (tid == 0) *done = 0;
        const auto at = [&](int i) { return (long long)slot_of(b + i * by) * kM; };
        for (int x = tid; x < live * count; x += NT) s.parts[x / live][x % live] = __ldcg(&p.part_ml[at(x / live) + x % live]);
        __syncthreads();
        constexpr int kPer = kM * D / 2 / NT, kAt = kPer < 4 ? kPer : 4;  // pairs of columns of a thread; at a time
#pragma unroll 1
        for (int x0 = tid; x0 < live * D / 2; x0 += kAt * NT) {
          float2 v[kAt];
          float top[kAt], sum[kAt];
#pragma unroll
          for (int k = 0; k < kAt; ++k) {
            v[k] = make_float2(0.f, 0.f);
            top[k] = -INFINITY;
            sum[k] = 0.f;
            for (int i = 0; i < count; ++i) top[k] = fmaxf(top[k], s.parts[i][(x0 + k * NT) / (D / 2) % kM].x);
          }
#pragma unroll 4
          for (int i = 0; i < count; ++i) {
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
              // rows past the live ones are read, and nobody's
              const int x = x0 + k * NT, r = x / (D / 2) % kM, c = 2 * (x % (D / 2));
              const float2 y = __ldcg(reinterpret_cast<const float2*>(p.part + (at(i) + r) * D + c)), ml = s.parts[i][r];
              const float e = ml.x == -INFINITY ? 0.f : ex2(ml.x - top[k]);
              sum[k] = fmaf(ml.y, e, sum[k]);
              v[k].x = fmaf(y.x, e, v[k].x);
              v[k].y = fmaf(y.y, e, v[k].y);
            }
          }
#pragma unroll
          for (int k = 0; k < kAt; ++k) {
            const int x = x0 + k * NT, r = x / (D / 2), c = 2 * (x % (D / 2));
            if (r >= live) break;
            if (level == 1) {
              put2<D>(p, w.row0, w.h, w.i * kM + r, c, v[k], sum[k]);
            } else {
              *reinterpret_cast<float2*>(p.part + (at(0) + r) * D + c) = v[k];
              if (c == 0) p.part_ml[at(0) + r] = make_float2(top[k], sum[k]);
            }
          }
        }
        __syncthreads();
      }
    }
    __syncthreads();
    if (step + 1 < steps) w.next_task();
    fresh = true;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!ok) {
    // A wait has passed its limit: the stages' last copies are waited for.
    for (int i = max(0, steps - ST); i < steps; ++i)
      if (boxed >> (i % ST) & 1) mbar_wait(&s.full[grp][i % ST], ~phases >> (i % ST) & 1);
    if (lane == 0) atomicCAS(p.error, 0u, (kStatusDeadline << 24) | (kAttnWait << 16) | (blockIdx.x & 0xffff));
  }
}

template <int D>
__global__ void __launch_bounds__(1024) plan_kernel(const AttnParams p) {
  __shared__ PlanScratch<1024> x;
  griddep_wait();
  griddep_launch_dependents();
  attn_plan<Rows<D>::kKT, 1024>(p, p.seq, p.start, x, true);
}

template <int D>
cudaError_t launch(AttnParams p, int grid, cudaStream_t s) {
  const size_t smem = sizeof(RowsSmem<D>);
  cudaError_t e = opt_in<attn_rows<D>>(smem);
  if (e != cudaSuccess) return e;
  if (p.seqs <= kAttnPlanned) p.seq = nullptr;
  p.tile_m = 16;
  p.tile_g = p.group;
  RowMaps m = {};
  const long long rows = (long long)p.num_blocks * p.block.d, cols = (long long)p.Hkv * D;
  m.boxes = p.block.d % 16 == 0 && rows > 0;
  if (m.boxes && (!attn_row_map(&m.k, p.k, rows, cols, p.ldk, 16) || !attn_row_map(&m.v, p.v, rows, cols, p.ldv, 16)))
    return cudaErrorInvalidValue;
  if (p.seq) {
    const Launch one(dim3(1), 1024, 0, true, s);
    e = cudaLaunchKernelEx(&one.cfg, plan_kernel<D>, p);
    if (e != cudaSuccess) return e;
  }
  const Launch all(dim3(grid), Rows<D>::kW * 32, smem, true, s);
  return cudaLaunchKernelEx(&all.cfg, attn_rows<D>, m, p);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnParams& p, int d, int grid, cudaStream_t s) {
  return d == 64 ? launch<64>(p, grid, s) : d == 128 ? launch<128>(p, grid, s) : launch<256>(p, grid, s);
}

}  // namespace gdn
