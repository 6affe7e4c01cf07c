// Paged attention (gdn_attn_paged) on the tensor cores (tcgen05): more query rows than
// gdn_attn_rows.cu takes at a time.
//
// A task is up to two tiles of 128 query rows (one of heads of 256) of a request and
// key/value head, the G query heads of a token next to one another, so that every key and value
// that comes into shared memory serves 256 rows. For each tile of keys
//   S = Q K^T (TMEM), P = 2^(scale log2(e) S - m) as bf16 (TMEM, over S), O += P V (TMEM),
// with m a maximum that follows the running one at a distance of up to 8: a row's O and sum are
// multiplied only when the maximum grows by more, so that weights are at most 2^8 and hardly a
// tile is corrected; the sums divide it out again.
//
// Warps 0 - 7: the softmax, a row a thread, and the outputs. Warps 8 - 11: keys and values by
// TMA, four rows a copy from any four slots (so blocks of any size are alike, and rows past the last key
// are zeros). Warp 12: the products. With two row tiles the tensor cores work on one while
// the softmax works on the other; with one, S alternates between two buffers.
#include <climits>

#include "gdn_attn.cuh"
#include "gdn_host.h"
#include "gdn_prefill.cuh"
#include "gdn_tc_pair.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kNT = 512;
constexpr int kLoad0 = 8, kMma = 12;  // first load warp; the warp of the products
constexpr float kSlack = 8.f;         // log2 of the most that a weight is above 1

template <int D>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;        // row tiles of a task
  static constexpr int kM = 128 * kTiles;
  static constexpr int kKT = D == 256 ? 64 : 128;        // keys of a tile
  static constexpr int kE = D == 256 ? 6 : 3;            // tiles' time that a task takes beside its tiles
  static constexpr int kSlots = D == 64 ? 8 : D == 128 ? 5 : 4;
  static constexpr int kSlotBytes = kKT * D * 2;         // 32 KB, 16 KB with heads of 64
  static constexpr int kChunk = kKT * 128;               // bytes of 64 columns of a slot
  // TMEM columns: S of the two row tiles, or S's two buffers; O
  static constexpr int kS = D == 256 ? 64 : 128;
  static constexpr int kO = 256;
};

template <int D>
struct alignas(1024) TileSmem {
  using C = Cfg<D>;
  unsigned char q[C::kTiles][128 * D * 2];
  unsigned char ring[C::kSlots][C::kSlotBytes];
  uint64_t q_full, q_empty, edge, full[C::kSlots], empty[C::kSlots], s_full[2], p_full[2], o_done[2], seg_done[2][2];
  uint32_t tmem;
  int failed;          // a wait has passed its limit
  unsigned last[2];
  int at[4];           // the first unit's request, head, row tile and key tile
  int dirty[2];        // whether there are any of
  int poison[2][D];    // by task: the first key, hidden from some row, whose value in the column is not finite
  int4 seq[kAttnPlannedTiles + 1];
  long long start[kAttnPlannedTiles + 1];
  PlanScratch<kNT> scan;
};

__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// Descriptor of an N-major operand in the 128-byte swizzled layout: K rows of 128 bytes (64 N
// values), 8-row groups 1024 bytes apart, the next 64 N values `next` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t next) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(next >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
constexpr uint32_t kMnB = 1u << 16;  // idesc: B is N-major

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two f32 at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// A barrier of some of the warps that also tells whether all of them are well: a warp whose
// wait has failed must not leave the others at one.
__device__ __forceinline__ bool named_all(int id, int threads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.and.pred b, %1, %2, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// 32 columns of a done row: divided by the sum, gated, stored.
__device__ __forceinline__ void put32(const AttnParams& p, long long row, long long col, const float (&v)[32], float inv) {
  __nv_bfloat16* o = p.out + row * p.ldo + col;
  uint32_t w[16];
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = v[c + j] * inv;
    if (p.gate) {
      const uint4 z = *reinterpret_cast<const uint4*>(p.gate + row * p.ldg + col + c);
      const uint32_t u[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = __fdividef(y[2 * j], 1.f + __expf(-bf16_lo(u[j])));
        y[2 * j + 1] = __fdividef(y[2 * j + 1], 1.f + __expf(-bf16_hi(u[j])));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[c / 2 + j] = pack2(y[2 * j], y[2 * j + 1]);
  }
  if (p.wide_out) {  // whole sectors: the lanes' rows are far from one another
#pragma unroll
    for (int c = 0; c < 2; ++c)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(o + 16 * c), "r"(w[8 * c]), "r"(w[8 * c + 1]),
                   "r"(w[8 * c + 2]), "r"(w[8 * c + 3]), "r"(w[8 * c + 4]), "r"(w[8 * c + 5]), "r"(w[8 * c + 6]), "r"(w[8 * c + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint4*>(o + 8 * c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
}

// The CTA's share as a walk of segments: what is left of a task, or as much of it as is the
// CTA's.
template <int D>
struct Segments {
  using C = Cfg<D>;
  Walk<C::kM, C::kKT, C::kE> w;
  long long u, u1;
  int j0, j1;  // key tiles of the segment
  __device__ __forceinline__ Segments(const AttnParams& p, const int4* seq, const long long* start, long long u0, long long u1,
                                      const int (&at)[4])
      : w(p, seq, start), u(u0), u1(u1) {
    w.from(at, u0);
    j0 = w.j;
    j1 = (int)min((long long)w.nt, j0 + (u1 - u));
    if (j0 >= w.nt) next();  // what the share begins with of a task has no tiles
  }
  // Whether there is a segment.
  __device__ __forceinline__ bool valid() const { return u < u1; }
  __device__ __forceinline__ bool next() {
    u = w.task + w.nt + C::kE;
    if (u >= u1) return false;
    w.next_task();
    j0 = 0;
    j1 = (int)min((long long)w.nt, u1 - u);
    return true;
  }
  // end of row tile t's key tiles in the segment: its last row may see fewer than the task's
  __device__ __forceinline__ int end(int t) const {
    const int rows = w.n * (int)w.p.group.d, first = w.i * C::kM + t * 128;
    if (first >= rows) return j0;
    const int last = min(first + 128, rows) - 1;
    return max(j0, min(j1, (w.ctx + (int)w.p.group.div(last) + C::kKT) / C::kKT));
  }
};

// The caches' rows as the copies want them: one at a time, and in boxes of `box` rows (0: no boxes).
struct TileMaps {
  CUtensorMap k, v, kb, vb;
  int box;
};
// Four rows of 64 columns from column x on, each of its own, to 512 bytes of shared memory.
__device__ __forceinline__ void gather4(void* dst, const CUtensorMap* map, int x, const int (&row)[4], uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(smem_u32(bar))
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(kNT, 1)
    attn_tiles(const __grid_constant__ TileMaps maps, const AttnParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  static_assert(sizeof(TileSmem<D>) <= 232448, "227 KB of shared memory a CTA");
  TileSmem<D>& s = *reinterpret_cast<TileSmem<D>*>(raw);
  constexpr int KT = C::kKT, SLOTS = C::kSlots;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&s.q_full, 4);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.edge, 4);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    if (maps.box) prefetch_tensormap(&maps.kb), prefetch_tensormap(&maps.vb);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&s.full[i], 4);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
      mbar_init(&s.o_done[i], 1);
      for (int t = 0; t < 2; ++t) mbar_init(&s.seg_done[t][i], 4);
    }
    s.failed = s.dirty[0] = s.dirty[1] = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < 2 * D; i += kNT) (&s.poison[0][0])[i] = INT_MAX;
  if (warp == kMma) tmem_alloc(&s.tmem, 512);
  griddep_wait();
  griddep_launch_dependents();
  const int4* seq = s.seq;
  const long long* start = s.start;
  if (p.seq) {
    seq = p.seq;
    start = p.start;
  } else {
    attn_plan<C::kM, KT, C::kE, kNT>(p, s.seq, s.start, s.scan, blockIdx.x == 0);
  }
  attn_zero_rows<kNT / 32>(p, seq, p.Hkv * p.group.d * D);
  const long long units = start[p.seqs];
  const Shares shares(units, (int)max(1LL, min((long long)gridDim.x, (units + C::kE + 1) / (C::kE + 2))));
  const bool on = units > 0 && blockIdx.x < shares.ctas;
  const long long u0 = shares.first(blockIdx.x), u1 = shares.first(blockIdx.x + 1);
  if (warp == 0 && on) Walk<C::kM, KT, C::kE>::find(p, seq, start, u0, s.at);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const int rows_end = p.num_blocks * (int)p.block.d;
  bool ok = on;

  if (warp < kLoad0) {
    more_regs<200>();
    const int t = warp >> 2;  // row tile
    if (ok && t < C::kTiles) {
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const int r = (warp & 3) * 32 + lane;
      Segments<D> g(p, seq, start, u0, u1, s.at);
      int sn = 0, pv = 0, ends = 0;  // S tiles, PV products and segments with any so far (of the row tile)
      int seg = 0;
      if (g.valid()) do {
        const int rows = g.w.n * (int)p.group.d, first = g.w.i * C::kM + t * 128, R = first + r;
        const bool live = R < rows, warp_live = first + (warp & 3) * 32 < rows;
        const int last_key = g.w.ctx + (int)p.group.div(min(R, rows - 1));
        const int end = g.end(t);
        float m = -INFINITY, l = 0.f;
        for (int j = g.j0; j < end && ok; ++j, ++sn) {
          const int b = C::kTiles == 2 ? t : sn & 1;
          const uint32_t sc = tmem + lanes + b * C::kS;
          ok = mbar_wait(&s.s_full[b], (C::kTiles == 2 ? sn : sn >> 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (warp_live) {
            float x[KT];
#pragma unroll
            for (int c = 0; c < KT; c += 32) tmem_ld32(sc + c, *reinterpret_cast<float(*)[32]>(x + c));
            const int seen = last_key - j * KT;  // the tile's keys 0 .. seen
            if (__any_sync(0xffffffffu, seen < KT - 1)) {
#pragma unroll
              for (int c = 0; c < KT; ++c)
                if (c > seen) x[c] = -INFINITY;
            }
            float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int c = 4; c < KT - 4; c += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) top[i] = max3(top[i], x[c + i], x[c + 4 + i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], x[KT - 4 + i]);
            const float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
            if (__any_sync(0xffffffffu, tile_top > m + kSlack || m == -INFINITY)) {
              const float grown = fmaxf(m, tile_top), f = m == -INFINITY ? 0.f : ex2(m - grown);
              if (j > g.j0) {
                if (C::kTiles == 1) {  // S came before the last PV
                  ok = mbar_wait(&s.o_done[(pv - 1) & 1], ((pv - 1) >> 1) & 1);
                  ok = __all_sync(0xffffffffu, ok);
                  if (!ok) break;
                  tc_fence_after();
                }
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  float o[32];
                  const uint32_t at = tmem + lanes + C::kO + t * D + c;
                  tmem_ld32(at, o);
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] *= f;
                  tmem_st32(at, reinterpret_cast<const uint32_t*>(o));
                }
              }
              l *= f;
              m = grown;
            }
            const float base = m == -INFINITY ? 0.f : m;
            const float2 by = make_float2(p.scale_log2, p.scale_log2), less = make_float2(-base, -base);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < KT; c += 64) {
              uint32_t w[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float2 y = fma2(make_float2(x[c + 2 * i], x[c + 2 * i + 1]), by, less);
                y.x = ex2(y.x);
                y.y = ex2(y.y);
                sum[i & 1] = add2(sum[i & 1], y);
                w[i] = pack2(y.x, y.y);
              }
              tmem_st32(sc + c / 2, w);
            }
            sum[0] = add2(sum[0], sum[1]);
            l += sum[0].x + sum[0].y;
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.p_full[b]);
          ++pv;
        }

        // ---- the task's end, or this CTA's
        const bool any = end > g.j0;
        if (any && ok) {
          ok = C::kTiles == 1 ? mbar_wait(&s.o_done[(pv - 1) & 1], ((pv - 1) >> 1) & 1) : mbar_wait(&s.o_done[t], ends++ & 1);
          tc_fence_after();
        }
        if (!(ok = named_all(1 + t, 128, ok))) break;
        const long long t0 = g.w.task, t1 = t0 + g.w.nt;
        const bool whole = t0 >= u0 && t1 <= u1;
        const long long slot = (2LL * blockIdx.x + (t0 >= u0)) * C::kM + t * 128;  // the part's first row
        const uint32_t tok = p.group.div(live ? R : 0), hd = (live ? R : 0) - tok * p.group.d;
        const long long row = g.w.row0 + tok, col = ((long long)g.w.h * p.group.d + hd) * D;
        const int* poison = s.poison[seg & 1];
        const bool flagged = any && s.dirty[seg & 1] != 0;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (warp_live) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            if (any) {
              tmem_ld32(tmem + lanes + C::kO + t * D + c, o);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (flagged && poison[c + i] <= last_key) o[i] = NAN;
            if (live) {
              if (whole) {
                put32(p, row, col + c, o, inv);
              } else {
                float4* part = reinterpret_cast<float4*>(p.part + slot * D) + c / 4 * 128 + r;
#pragma unroll
                for (int i = 0; i < 32; i += 4) part[i / 4 * 128] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
              }
            }
          }
          if (!whole && live) p.part_ml[slot + r] = make_float2(m, l);
        }
        __syncwarp();
        if (lane == 0 && any) mbar_arrive(&s.seg_done[t][seg & 1]);
        if (!whole && first < rows) {
          const int c0 = shares.owner(t0), c1 = shares.owner(t1 - 1);
          __threadfence();
          named_sync(1 + t, 128);
          if (r == 0) {
            s.last[t] = atomicAdd(p.done + 2 * c0 + t, 1u) == (unsigned)(c1 - c0);
            __threadfence();
          }
          named_sync(1 + t, 128);
          if (s.last[t]) {
            // every part is there: the first CTA's second one, the others' first
            if (r == 0) p.done[2 * c0 + t] = 0;
            const auto at = [&](int c) { return (2LL * c + (c == c0)) * C::kM + t * 128; };
            float top = -INFINITY, sum = 0.f;
            if (live) {
#pragma unroll 4
              for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(&p.part_ml[at(c) + r]).x);
#pragma unroll 4
              for (int c = c0; c <= c1; ++c) {
                const float2 ml = __ldcg(&p.part_ml[at(c) + r]);
                sum += ml.y * (ml.x == -INFINITY ? 0.f : ex2(ml.x - top));
              }
              const float in = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
              for (int k = 0; k < D; k += 32) {
                float o[32] = {};
#pragma unroll 2
                for (int c = c0; c <= c1; ++c) {
                  const float pm = __ldcg(&p.part_ml[at(c) + r]).x, e = pm == -INFINITY ? 0.f : ex2(pm - top);
                  const float4* part = reinterpret_cast<const float4*>(p.part + at(c) * D) + k / 4 * 128 + r;
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const float4 v = __ldcg(part + i * 128);
                    o[4 * i] = fmaf(v.x, e, o[4 * i]);
                    o[4 * i + 1] = fmaf(v.y, e, o[4 * i + 1]);
                    o[4 * i + 2] = fmaf(v.z, e, o[4 * i + 2]);
                    o[4 * i + 3] = fmaf(v.w, e, o[4 * i + 3]);
                  }
                }
                put32(p, row, col + k, o, in);
              }
            }
          }
        }
        ++seg;
      } while (g.next());
    }
  } else {
    fewer_regs<56>();
    if (warp < kMma) {
      // ---- keys, values and queries
      const int wl = warp - kLoad0, lt = tid - kLoad0 * 32;
      constexpr int kKeys = KT / 4;           // keys of a warp
      constexpr int kFours = kKeys / 4;       // of them four a copy, 64 columns wide: a lane each
      constexpr uint32_t kShare = kKeys * D * 2;
      static_assert(kFours * (D / 64) <= 32, "one copy a lane");
      const int four = lane % kFours, chunk = lane / kFours;
      const bool issues = chunk < D / 64;
      const uint32_t place = chunk * C::kChunk + (wl * kKeys + four * 4) * 128;
      // Where blocks are made of boxes of 8 rows or more, a whole tile comes as boxes: a copy of four
      // rows takes an SM 22 cycles whatever its size.
      const int boxes = min(maps.box, kKeys) > 0 ? kKeys / min(maps.box, kKeys) : 0;  // of a warp's keys, 64 columns wide
      const int box_chunk = boxes ? lane / boxes : 0, box_row = boxes ? lane % boxes * (kKeys / boxes) : 0;
      const bool box_issues = box_chunk < D / 64;
      const uint32_t box_place = box_chunk * C::kChunk + (wl * kKeys + box_row) * 128;
      int n = 0;                      // slots filled
      uint32_t edges = 0;             // edge tiles so far
      const auto wait = [&](uint64_t* b, uint32_t parity) { return ok = __all_sync(0xffffffffu, mbar_wait(b, parity)); };
      if (ok) {
        Segments<D> g(p, seq, start, u0, u1, s.at);
        int seg = 0;
        uint32_t waits[2] = {0, 0}, phases[2] = {0, 0};  // by row tile, a bit for even and odd tasks
        if (g.valid()) do {
          if (seg >= 2) {
            // The flags are the task's before last until its row tiles are through with them. (A row
            // tile without keys in a segment says nothing: nothing would keep it from running ahead.)
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t)
              if (waits[t] >> (seg & 1) & 1) {
                ok = ok && wait(&s.seg_done[t][seg & 1], phases[t] >> (seg & 1) & 1);
                phases[t] ^= 1u << (seg & 1);
              }
            if (!(ok = named_all(3, 128, ok))) break;
            const bool flagged = s.dirty[seg & 1] != 0;
            named_sync(3, 128);
            if (flagged) {
              for (int i = lt; i < D; i += 128) s.poison[seg & 1][i] = INT_MAX;
              if (lt == 0) s.dirty[seg & 1] = 0;
              named_sync(3, 128);
            }
          }
#pragma unroll
          for (int t = 0; t < C::kTiles; ++t)
            waits[t] = (waits[t] & ~(1u << (seg & 1))) | (uint32_t)(g.end(t) > g.j0) << (seg & 1);
          const int keys = g.w.ctx + g.w.n, first_last = g.w.ctx + (int)p.group.div(g.w.i * C::kM);
          const int x = g.w.h * D + chunk * 64, box_x = g.w.h * D + box_chunk * 64;
          // a lane has the slot of one of the warp's keys, a tile ahead
          KeyBlock kb = key_block(p, g.w.s, g.j0 * KT + wl * kKeys + lane % kKeys, keys);
#pragma unroll 1
          for (int j = g.j0; j < g.j1 && ok; ++j) {
            int at[4], box_at;
            {
              const int slot = key_slot(p, kb, g.w.s), row = slot < 0 ? rows_end : slot;  // past the last row: zeros
#pragma unroll
              for (int i = 0; i < 4; ++i) at[i] = __shfl_sync(0xffffffffu, row, four * 4 + i);
              box_at = __shfl_sync(0xffffffffu, row, box_row);
            }
            if (j + 1 < g.j1) kb = key_block(p, g.w.s, (j + 1) * KT + wl * kKeys + lane % kKeys, keys);
#pragma unroll 1
            for (int which = 0; which < 2; ++which, ++n) {  // keys, values
              if (!wait(&s.empty[n % SLOTS], (n / SLOTS & 1) ^ 1)) break;
              unsigned char* to = s.ring[n % SLOTS];
              // some row does not see some of these keys
              const bool edge = which && j * KT + KT - 1 > first_last && g.w.n > 1;
              uint64_t* bar = edge ? &s.edge : &s.full[n % SLOTS];
              if (lane == 0) mbar_arrive_expect_tx(bar, kShare);
              __syncwarp();
              if (boxes && (j + 1) * KT <= keys) {
                if (box_issues) tma_load_2d_plain(to + box_place, which ? &maps.vb : &maps.kb, box_x, box_at, bar);
              } else if (issues) {
                gather4(to + place, which ? &maps.v : &maps.k, x, at, bar);
              }
              if (edge) {
                // 0 x NaN: values that are not finite are taken out, and the rows that do see them told
                // by the column's first such key
                if (!wait(&s.edge, edges++ & 1)) break;
                bool found = false;
                constexpr int kRow = D / 8;  // 16-byte pieces
#pragma unroll 4
                for (int i = lane; i < kKeys * kRow; i += 32) {
                  const int row = wl * kKeys + i / kRow, c = i % kRow;
                  const uint4 v = *reinterpret_cast<const uint4*>(to + (c >> 3) * C::kChunk + row * 128 + (((c ^ row) & 7) << 4));
                  // an exponent of ones, and one, is a carry into the sign's place
                  const auto not_finite = [](uint32_t u) { return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                  found |= (not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w)) != 0;
                }
                found = __any_sync(0xffffffffu, found);
                if (found) {
#pragma unroll 1
                  for (int i = lane; i < kKeys * D; i += 32) {
                    const int row = wl * kKeys + i / D, c = i % D;
                    uint16_t* q = reinterpret_cast<uint16_t*>(to + (c >> 6) * C::kChunk + row * 128 + ((((c >> 3) ^ row) & 7) << 4)) + (c & 7);
                    if ((*q & 0x7f80) == 0x7f80) {
                      atomicMin(&s.poison[seg & 1][c], j * KT + row);
                      *q = 0;
                    }
                  }
                }
                if (found) {
                  s.dirty[seg & 1] = 1;
                  fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.full[n % SLOTS]);
              }
              if (j == g.j0 && which == 0) {
                // the task's queries, beside its first keys; rows past the last are zero
                if (!wait(&s.q_empty, (seg & 1) ^ 1)) break;
                const int rows = g.w.n * (int)p.group.d;
                constexpr int kPieces = D / 8;  // 16-byte pieces of a row
                constexpr int kPer = 128 / kPieces;  // rows at once
                const int cc = lt % kPieces, base = g.w.i * C::kM;
                const uint32_t to_q = smem_u32(s.q[0]) + (cc >> 3) * (128 * 128);
                const __nv_bfloat16* from = p.q + g.w.row0 * p.ldq + (long long)g.w.h * p.group.d * D + cc * 8;
#pragma unroll 8
                for (int r0 = 0; r0 < C::kM; r0 += kPer) {
                  const int row = r0 + lt / kPieces, rr = row & 127;
                  const bool live = base + row < rows;
                  const uint32_t R = live ? base + row : 0, tok = p.group.div(R), hd = R - tok * p.group.d;
                  cp_async16_or_zero(to_q + (row >> 7) * (128 * D * 2) + rr * 128 + (((cc ^ rr) & 7) << 4),
                                     from + tok * p.ldq + hd * D, live);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.q_full);
                // the next ones on their way to L2
                if (g.u + (g.w.nt - g.w.j) + C::kE < u1 && base + C::kM < rows) {
#pragma unroll 2
                  for (int i = lt; i < C::kM * (D / 64); i += 128) {
                    const int R = base + C::kM + i / (D / 64);
                    if (R < rows) {
                      const uint32_t tok = p.group.div(R), hd = R - tok * p.group.d;
                      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + (g.w.row0 + tok) * p.ldq +
                                                                    ((long long)g.w.h * p.group.d + hd) * D + i % (D / 64) * 64));
                    }
                  }
                }
              }
            }
          }
          ++seg;
          ok = named_all(3, 128, ok);
        } while (ok && g.next());
        // No copy in flight when the CTA leaves: every slot that was filled is waited for. (A wait has
        // failed: the last phases that were begun.)
        for (int i = max(0, n - SLOTS); i < n; ++i) mbar_wait(&s.full[i % SLOTS], i / SLOTS & 1);
      }
    } else if (warp == kMma && ok) {
      // ---- the products
      Segments<D> g(p, seq, start, u0, u1, s.at);
      constexpr uint32_t is = idesc_bf16_f32(128, KT), io = idesc_bf16_f32(128, D) | kMnB;
      int n = 0, seg = 0, sn = 0, pn[2] = {0, 0};  // slots, tasks, S tiles (with one row tile), weights' tiles
      const auto wait = [&](uint64_t* b, uint32_t parity) {
        ok = ok && mbar_wait(b, parity);
        tc_fence_after();
      };
      // descriptors of the operands, as their low words change
      const uint64_t qd = sdesc_k_sw128(smem_u32(s.q[0])), kd = sdesc_k_sw128(smem_u32(s.ring[0])),
                     vd = sdesc_mn_sw128(smem_u32(s.ring[0]), C::kChunk);
      // S of row tile t (into buffer b) from the keys in ring slot k
      const auto scores = [&](int t, int b, int k) {
        const uint64_t a = qd + t * (128 * D * 2 >> 4), kk = kd + k * (C::kSlotBytes >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_bf16(tmem + b * C::kS, a + ((i >> 2) * (128 * 128) >> 4) + 2 * (i & 3), kk + ((i >> 2) * C::kChunk >> 4) + 2 * (i & 3),
                   is, i > 0);
        mma_commit(&s.s_full[b]);
      };
      const auto values = [&](int t, int b, int k, bool first, bool tell) {
        const uint64_t v = vd + k * (C::kSlotBytes >> 4);
#pragma unroll
        for (int i = 0; i < KT / 16; ++i)
          mma_bf16_ts(tmem + C::kO + t * D, tmem + b * C::kS + 8 * i, v + i * (2048 >> 4), io, !(first && i == 0));
        if (tell) mma_commit(&s.o_done[C::kTiles == 2 ? t : b]);
      };
      const auto filled = [&](int slot, int i) { wait(&s.full[slot], i / SLOTS & 1); };
      const auto after = [&](int slot, int d) { return slot + d >= SLOTS ? slot + d - SLOTS : slot + d; };
      int ks = 0;  // ring slot n % SLOTS: step i's keys are slot n + 2 i, its values n + 2 i + 1
      if (g.valid()) do {
        const int e[2] = {g.end(0), C::kTiles == 2 ? g.end(1) : g.j0};
        const int steps = g.j1 - g.j0;
        wait(&s.q_full, seg & 1);
        filled(ks, n);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (elect_one()) {
          if (C::kTiles == 2) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
              if (e[t] > g.j0) scores(t, t, ks);
          } else {
            scores(0, sn & 1, ks);
          }
          mma_commit(&s.empty[ks]);
          if (steps == 1) mma_commit(&s.q_empty);
        }
        __syncwarp();
        ++sn;
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
          const int vs = after(ks, 1), k2 = after(ks, 2), j = g.j0 + i;
          const bool more = i + 1 < steps;
          if (C::kTiles == 2) {
            // a row tile's softmax runs while the other's products do
            filled(vs, n + 1);
            if (more) filled(k2, n + 2);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const bool pv = j < e[t], s_ = j + 1 < e[t];
              if (pv) {
                wait(&s.p_full[t], pn[t] & 1);
                ++pn[t];
              }
              if (!(ok = __all_sync(0xffffffffu, ok))) break;
              if (elect_one()) {
                if (pv) values(t, t, vs, i == 0, !s_);
                if (t == 1) mma_commit(&s.empty[vs]);
                if (s_) scores(t, t, k2);
                if (t == 1 && more) mma_commit(&s.empty[k2]);
                if (t == 1 && i + 2 == steps) mma_commit(&s.q_empty);
              }
              __syncwarp();
            }
            if (!ok) break;
          } else {
            // S's buffers alternate over the whole share: the softmax of a tile runs beside the next one's S
            if (more) {
              filled(k2, n + 2);
              if (!(ok = __all_sync(0xffffffffu, ok))) break;
              if (elect_one()) {
                scores(0, sn & 1, k2);
                mma_commit(&s.empty[k2]);
                if (i + 2 == steps) mma_commit(&s.q_empty);
              }
              __syncwarp();
              ++sn;
            }
            const int b = pn[0] & 1;
            filled(vs, n + 1);
            wait(&s.p_full[b], (pn[0] >> 1) & 1);
            ++pn[0];
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            if (elect_one()) {
              values(0, b, vs, i == 0, true);
              mma_commit(&s.empty[vs]);
            }
            __syncwarp();
          }
          ks = k2;
          n += 2;
        }
        ++seg;
      } while (ok && g.next());
    }
  }
  if (on && !ok) {
    s.failed = 1;
    atomicCAS(p.error, 0u, (kStatusDeadline << 24) | (kAttnWait << 16) | (blockIdx.x & 0xffff));
  }
  tc_fence_before();
  // every role is through: the softmax has waited for the last products, or a wait has failed
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) {
    // a wait has failed somewhere: the products in flight take microseconds
    if (on && s.failed)
      for (int i = 0; i < 8; ++i) __nanosleep(1000000);
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
__global__ void __launch_bounds__(1024) plan_kernel(const AttnParams p) {
  __shared__ PlanScratch<1024> x;
  griddep_wait();
  griddep_launch_dependents();
  attn_plan<Cfg<D>::kM, Cfg<D>::kKT, Cfg<D>::kE, 1024>(p, p.seq, p.start, x, true);
}

// Tile map of a cache's rows: boxes of 64 columns, 128-byte swizzle, zeros past the last row.
bool row_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld, int box_rows) {
  typedef CUresult (*Fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                         const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                         CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Fn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (Fn)f;
  }();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(AttnParams p, int grid, cudaStream_t s) {
  const size_t smem = sizeof(TileSmem<D>);
  cudaError_t e = opt_in<attn_tiles<D>>(smem);
  if (e != cudaSuccess) return e;
  TileMaps m = {};
  const long long rows = (long long)p.num_blocks * p.block.d, cols = (long long)p.Hkv * D;
  // the largest power of two of rows that blocks are made of, up to a load warp's keys
  for (int b = 8; b <= Cfg<D>::kKT / 4 && p.block.d % b == 0; b *= 2) m.box = b;
  if (!row_map(&m.k, p.k, rows, cols, p.ldk, 1) || !row_map(&m.v, p.v, rows, cols, p.ldv, 1)) return cudaErrorInvalidValue;
  if (m.box && (!row_map(&m.kb, p.k, rows, cols, p.ldk, m.box) || !row_map(&m.vb, p.v, rows, cols, p.ldv, m.box)))
    return cudaErrorInvalidValue;
  if (p.seqs <= kAttnPlannedTiles) p.seq = nullptr;
  if (p.seq) {
    const Launch one(dim3(1), 1024, 0, true, s);
    e = cudaLaunchKernelEx(&one.cfg, plan_kernel<D>, p);
    if (e != cudaSuccess) return e;
  }
  const Launch all(dim3(grid), kNT, smem, true, s);
  return cudaLaunchKernelEx(&all.cfg, attn_tiles<D>, m, p);
}

}  // namespace

cudaError_t launch_attn_tiles(const AttnParams& p, int d, int grid, cudaStream_t s) {
  return d == 64 ? launch<64>(p, grid, s) : d == 128 ? launch<128>(p, grid, s) : launch<256>(p, grid, s);
}

}  // namespace gdn
