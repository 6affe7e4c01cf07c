// Paged attention (gdn_attn_paged) on the tensor cores (tcgen05): more query rows than
// gdn_attn_rows.cu takes at a time.
//
// Two CTAs work together (cta_group::2). A task is up to four tiles of 128 query rows (two with heads
// of 256), half of them each CTA's, of a request and key/value head: a tile holds as many tokens
// as fit with all their G heads. Every key and value that comes into the pair's shared memory,
// half of it in each CTA, serves all of them. For each tile of 128 keys
//   S = Q K^T (TMEM), P = 2^(scale log2(e) S - m) as bf16 (TMEM, over S), O += P V (TMEM),
// with m a maximum that follows the running one at a distance of up to 8: a row's O and sum are
// multiplied only when the maximum grows by more, so that weights are at most 2^8 and hardly a
// tile is corrected; the sums divide it out again.
//
// Warps 0 - 7: the softmax, a row a thread, and the outputs. Warps 8 - 11: queries, keys and values by
// TMA; the blocks' rows in boxes where a block is made of boxes of 8 or more, else four rows a copy
// from any four slots, and rows past the last key are zeros. Warp 12 of the first CTA: the
// products of both. Warp 13: which part of which task comes next. With two row tiles a CTA
// the tensor cores work on one while the softmax works on the other; with one, S alternates
// between two buffers. A task whose rows fill one tile of each CTA alone has the keys of
// every second tile in the place of the other tile's rows, and joins the two.
//
// Measured: chunks of 2048 tokens in all of two requests over up to 30000, 24 heads of 256 on 4, 757 - 795 us in bursts of ten
// (1.6 - 1.7 PFLOP/s, 84 - 88% of the measured burst rate; one CTA by itself, keys and values for 128 rows, 1460), 887 - 938 in
// a row of calls at the power limit (1.37 - 1.45 PFLOP/s, 79 - 84% of the measured sustained rate): the tensor cores. 8192 fresh
// tokens of 5 requests, 64 heads of 128 on 8, 275 us (64% of the burst rate; up to 394 right after such a row of chunks): a
// turn's products take 1080 cycles, but the chain S, softmax, PV of
// a row tile 3900, in which two turns run, as S and O fill TMEM. 24 requests of 4 tokens over up to 6000, 40 heads of
// 128 on 8, 73 us (57% of the bandwidth): 20 of a tile's 128 rows are there, each tile of keys is a turn all
// the same, and a task has 8 us of queries, first tile and join.
#include <algorithm>
#include <climits>

#include "gdn_attn.cuh"
#include "gdn_host.h"
#include "gdn_prefill.cuh"
#include "gdn_tc_pair.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kNT = 512;
constexpr int kLoad0 = 8, kMma = 12, kSched = 13;  // first load warp; the warp of the products; of the tasks
constexpr float kSlack = 8.f;                      // log2 of the most that a weight is above 1
constexpr int KT = 128;                            // keys of a tile
constexpr int kSegs = 4;                           // parts of tasks that are known ahead
// Key tiles from which on a task is split between a CTA's row tiles. With 4, 16, never (us; 2 and 8 as 4): 24 requests of 4
// tokens over up to 6000, 40 heads of 128 on 8, 68, 82, 100; 48 of 3 over up to 3000, 64 on 8, 88, 110, 120; 96 of 4 over up
// to 1000, 40 on 8, 102, 107, 108; 12 of 8 over up to 12000, 32 heads of 64 on 4, 37, 38, 52; but 8 of 16 over up to 30000, 8 on
// 1, 65, 66, 52.
constexpr int kSplit = 4;

template <int D>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;          // row tiles of a CTA
  static constexpr int kRows = 256 * kTiles;               // rows of a task
  static constexpr int kVCols = D == 256 ? 128 : 64;       // a CTA's columns of the values (heads of 64: 32, and 32 for nothing)
  static constexpr int kSlotBytes = D == 256 ? 32768 : 16384;  // 64 keys, or kVCols columns of 128 values
  static constexpr int kSlots = D == 64 ? 8 : D == 128 ? 9 : 4;
  static constexpr int kO = 256;                           // TMEM column of O; S of the two row tiles, or S's two buffers, before it
};

// A part of a task: what both CTAs of a pair, and all roles, work on next.
struct Seg {
  int s, h;        // request, key/value head
  int row0, toks;  // first row of the task's tokens, and how many
  int pos, keys;   // position of the first; the request's keys
  int j0, j1;      // key tiles
  int end[2];      // where those end that the row tiles of both CTAs see
  int c0, c1;      // pairs that work on the task
  int whole, slot; // nobody else does; which of the pair's two parts it is
  int split;       // the keys are split between the CTA's row tiles
  int on;          // 0: there is none
  unsigned tag;    // numbers the segments
};

template <int D>
struct alignas(1024) TileSmem {
  using C = Cfg<D>;
  unsigned char q[C::kTiles][128 * D * 2];
  unsigned char ring[C::kSlots][C::kSlotBytes];
  uint64_t q_full, q_empty, edge, full[C::kSlots], empty[C::kSlots], s_full[2], p_full[2], o_done[2], joined, seg_full[kSegs],
      seg_empty[kSegs];
  uint32_t tmem;
  int failed;                   // a wait has passed its limit
  unsigned last[2];
  float2 joint[C::kTiles][128];  // a joined row's maximum, and one over its sum
  unsigned split_done;          // row tiles that have finished their half of the keys of a task that is the pair's alone
  int at[4];                    // the first unit's request, head, row tile and key tile
  Seg seg[kSegs];
  // By segment: the first key, hidden from some row, whose value in the column is not finite, as
  // (tag << 12 | 4095 - the key's distance from pos), so that what is left of another segment is none; whether
  // there are any: the tag.
  unsigned poison[kSegs][D], flagged[kSegs];
  int4 plan[kAttnPlanned + 1];
  long long start[kAttnPlanned + 1];
  PlanScratch<kNT> scan;
};

// D[both CTAs' tmem] (+)= A[both CTAs' tmem] B, 256 rows; half of B in each CTA.
__device__ __forceinline__ void mma_bf16_ts_pair(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
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

// On a barrier of either CTA (its cluster address). Not releases at cluster scope: those wait for all that the
// thread has written, a thousand cycles with each tile; what these two tell of is in TMEM, behind
// tcgen05's own fences, or on its way by TMA.
__device__ __forceinline__ void arrive_expect_cluster(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void atomic_max_cluster(uint32_t at, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
// Four rows of 64 columns from column x on, each of its own, to 512 bytes of this CTA's shared memory; `bar` of either CTA.
__device__ __forceinline__ void gather4_pair(void* dst, const CUtensorMap* map, int x, const int (&row)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

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
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t (&r)[32]) {
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

// The caches' rows as the copies want them: one at a time, and in boxes of box_k and box_v rows (0: no
// boxes); the queries' as a row tile's tokens with their heads.
struct TileMaps {
  CUtensorMap k, v, kb, vb, q;
  int box_k, box_v;
  int tokens;  // of a row tile
};

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kNT, 1)
    attn_tiles(const __grid_constant__ TileMaps maps, const AttnParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  static_assert(sizeof(TileSmem<D>) <= 232448, "227 KB of shared memory a CTA");
  TileSmem<D>& s = *reinterpret_cast<TileSmem<D>*>(raw);
  constexpr int SLOTS = C::kSlots, TILES = C::kTiles;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    mbar_init(&s.q_full, 2);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.edge, 2);
    mbar_init(&s.joined, 8);
    s.split_done = 0;
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&s.full[i], 4);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 8);
      mbar_init(&s.o_done[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&s.seg_full[i], 1);
      mbar_init(&s.seg_empty[i], 8 * TILES + 4 + (rank == 0));  // both CTAs' softmax, the load warps, the products
      s.flagged[i] = 0;
    }
    s.failed = 0;
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    if (maps.box_k) prefetch_tensormap(&maps.kb), prefetch_tensormap(&maps.vb);
    prefetch_tensormap(&maps.q);
    fence_mbar_init();
  }
  for (int i = tid; i < kSegs * D; i += kNT) (&s.poison[0][0])[i] = 0;
  if (warp == kMma) tmem_alloc_pair(&s.tmem, 512);
  griddep_wait();
  griddep_launch_dependents();
  const int4* plan = s.plan;
  const long long* start = s.start;
  if (p.seq) {
    plan = p.seq;
    start = p.start;
  } else {
    attn_plan<KT, kNT>(p, s.plan, s.start, s.scan, blockIdx.x == 0);
  }
  attn_zero_rows<kNT / 32>(p, plan, p.Hkv * p.group.d * D);
  const long long units = start[p.seqs];
  const Shares shares(units, (int)max(1LL, min((long long)pairs, (units + p.tile_e + 1) / (p.tile_e + 2))));
  const bool on = units > 0 && pair < shares.ctas;
  const long long u0 = shares.first(pair), u1 = shares.first(pair + 1);
  if (warp == kSched && on) Walk<KT>::find(p, plan, start, u0, s.at);
  __syncthreads();
  cluster_sync();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const int G = p.group.d, tile_toks = maps.tokens, rows_end = p.num_blocks * (int)p.block.d;
  bool ok = on;
  // The next segment, by its number.
  const auto take = [&](int n) {
    ok = ok && mbar_wait(&s.seg_full[n % kSegs], n / kSegs & 1);
    ok = __all_sync(0xffffffffu, ok);
    return ok && s.seg[n % kSegs].on;
  };

  if (warp < kLoad0) {
    more_regs<192>();
    const int t = warp >> 2;  // row tile
    if (t < TILES) {
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const int r = (warp & 3) * 32 + lane;
      const bool in_tile = r < tile_toks * G, warp_in_tile = (warp & 3) * 32 < tile_toks * G;
      const int r_tok = p.group.div(r), hd = r - r_tok * G, warp_tok = p.group.div((warp & 3) * 32);
      int sn = 0, ends = 0, joins = 0;  // S tiles, segments with any so far (of the row tile), split tasks that are the pair's alone
      for (int n = 0;; ++n) {
        const bool there = take(n);
        if (!(ok = named_all(1 + t, 128, ok)) || !there) break;
        const Seg& g = s.seg[n % kSegs];
        const bool split = TILES == 2 && g.split;
        const int j0 = g.j0 + (split ? t : 0), end = g.end[t], step = split ? 2 : 1, toks = g.toks, pos = g.pos;
        const int first = ((split ? 0 : 2 * t) + rank) * tile_toks, tok = first + r_tok;  // the tile's first token, the row's
        const bool live = in_tile && tok < toks, warp_live = warp_in_tile && first + warp_tok < toks;
        const int last_key = pos + min(tok, toks - 1);
        float m = -INFINITY, l = 0.f, by1 = p.scale_log2, less1 = 0.f;  // weights are 2^(x by1 + less1)
#pragma unroll 1
        for (int j = j0; j < end; j += step, ++sn) {
          const int b = TILES == 2 ? t : sn & 1;
          const uint32_t sc = tmem + lanes + b * 128;
          ok = mbar_wait(&s.s_full[b], (TILES == 2 ? sn : sn >> 1) & 1);
          tc_fence_after();
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
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
            const float largest = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), tile_top = largest * p.scale_log2;
            // rows that are none have what was in their place: their maxima correct nothing
            if (__any_sync(0xffffffffu, live && (tile_top > m + kSlack || m == -INFINITY))) {
              const float grown = fmaxf(m, tile_top), f = m == -INFINITY ? 0.f : ex2(m - grown);
              if (j > j0) {
                if (TILES == 1) {  // S came before the last PV
                  ok = mbar_wait(&s.o_done[(sn - 1) & 1], ((sn - 1) >> 1) & 1);
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
                  uint32_t w[32];
#pragma unroll
                  for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i]);
                  tmem_st32(at, w);
                }
              }
              l *= f;
              // x scale - m in one rounding is off by what m was rounded by: a factor of all weights, which their sum has too, but
              // from scores of 2^31 on one that passes f32's range. There the next smaller score is at least 64 below, and
              // a power of two for the scale, which rounds nothing, tells the largest one from all others as well.
              if (tile_top > m) {
                const bool far = fabsf(tile_top) >= 0x1p30f;
                by1 = far ? p.scale_pow2 : p.scale_log2;
                less1 = far ? -(largest * by1) - (tile_top - tile_top) : -tile_top;
              }
              m = grown;
            }
            const float2 by = make_float2(by1, by1), less = make_float2(less1, less1);
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
          if (lane == 0) arrive_cluster(map_rank(&s.p_full[b], 0));
        }

        // ---- the task's end, or this pair's
        const bool any = end > j0;
        if (any && ok) {
          // with two row tiles O is told done once a segment, with one for every tile
          ok = TILES == 1 ? mbar_wait(&s.o_done[(sn - 1) & 1], ((sn - 1) >> 1) & 1) : mbar_wait(&s.o_done[t], ends & 1);
          ++ends;
          tc_fence_after();
        }
        if (!(ok = named_all(1 + t, 128, ok))) break;
        const int c0 = g.c0, c1 = g.c1;
        const bool own = g.whole, whole = own && !split;
        const long long part_row = (2LL * pair + g.slot) * C::kRows + (2 * t + rank) * 128;  // the part's first row
        const long long row = g.row0 + tok, col = ((long long)g.h * G + hd) * D;
        const int g_row0 = g.row0, g_h = g.h;
        const unsigned tag = g.tag;
        const unsigned* poison = s.poison[n % kSegs];
        const bool flagged = __any_sync(0xffffffffu, any && s.flagged[n % kSegs] == tag);
        // The segment's entry and flags are free once both CTAs' softmax has read them: this CTA writes the next one's entry
        // over them, either its flags. Where there are no flags the other CTA need not wait for a read, as whatever
        // it writes is not this tag; a release at cluster scope costs half a microsecond a segment.
        if (!flagged) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.seg_empty[n % kSegs]);
          if (lane == 1) arrive_cluster(map_rank(&s.seg_empty[n % kSegs], rank ^ 1));
        }
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
            if (flagged) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const unsigned q = poison[c + i];
                if (q >> 12 == tag && (int)(4095 - (q & 4095)) <= last_key - pos + 1024) o[i] = NAN;
              }
            }
            if (live) {
              if (whole) {
                put32(p, row, col + c, o, inv);
              } else {
                float4* part = reinterpret_cast<float4*>(p.part + part_row * D) + c / 4 * 128 + r;
#pragma unroll
                for (int i = 0; i < 32; i += 4) part[i / 4 * 128] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
              }
            }
          }
          if (!whole && live) p.part_ml[part_row + r] = make_float2(m, l);
        }
        if (flagged) {
          __syncwarp();
          if (lane < 2) mbar_arrive_cluster(map_rank(&s.seg_empty[n % kSegs], lane));
        }
        if (!whole && first < toks) {
          // A task that is the pair's alone, and split, is counted here: the counter in memory is that of the task
          // that other pairs go on with, who may be there long before this one.
          const bool alone = split && own;
          unsigned* done = p.done + 4 * c0 + (split ? 0 : 2 * t) + rank;
          const int parts = (c1 - c0 + 1) << (split ? 1 : 0);
          named_sync(1 + t, 128);
          if (r == 0) {
            unsigned before;
            if (alone) {
              __threadfence();
              before = atomicAdd(&s.split_done, 1u);
              __threadfence();
            } else {
              before = atom_add_acq_rel_u32(done, 1u);
            }
            s.last[t] = before == (unsigned)(parts - 1);
          }
          named_sync(1 + t, 128);
          if (s.last[t]) {
            // every part is there: the first pair's second one, the others' first, and where the keys
            // are split both row tiles'
            if (r == 0) {
              if (alone)
                s.split_done = 0;
              else
                *done = 0;
            }
            const auto at = [&](int k) {
              const int c = c0 + (split ? k >> 1 : k), u = split ? k & 1 : t;
              return (2LL * c + (c == c0)) * C::kRows + (2 * u + rank) * 128;
            };
            // a row a thread: the parts' maximum and sum; then 32 columns of a row a thread, whichever rows there are
            const int rows = min(tile_toks, toks - first) * G;
            if (r < rows) {
              float top = -INFINITY, sum = 0.f;
#pragma unroll 8
              for (int k = 0; k < parts; ++k) {
                const float2 ml = __ldcg(&p.part_ml[at(k) + r]);
                const float grown = fmaxf(top, ml.x);
                sum = sum * (top == -INFINITY ? 0.f : ex2(top - grown)) + ml.y * (ml.x == -INFINITY ? 0.f : ex2(ml.x - grown));
                top = grown;
              }
              s.joint[t][r] = make_float2(top, sum == 0.f ? 0.f : 1.f / sum);
            }
            named_sync(1 + t, 128);
#pragma unroll 1
            for (int e = r; e < rows * (D / 32); e += 128) {
              const int c = e / rows, i = e - c * rows, i_tok = p.group.div(i);
              const float2 joint = s.joint[t][i];
              float o[32] = {};
#pragma unroll 2
              for (int k = 0; k < parts; ++k) {
                const float pm = __ldcg(&p.part_ml[at(k) + i]).x, w = pm == -INFINITY ? 0.f : ex2(pm - joint.x);
                const float4* part = reinterpret_cast<const float4*>(p.part + at(k) * D) + c * 8 * 128 + i;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  const float4 v = __ldcg(part + q * 128);
                  o[4 * q] = fmaf(v.x, w, o[4 * q]);
                  o[4 * q + 1] = fmaf(v.y, w, o[4 * q + 1]);
                  o[4 * q + 2] = fmaf(v.z, w, o[4 * q + 2]);
                  o[4 * q + 3] = fmaf(v.w, w, o[4 * q + 3]);
                }
              }
              put32(p, g_row0 + first + i_tok, ((long long)g_h * G + i - i_tok * G) * D + 32 * c, o, joint.y);
            }
          }
        }
        if (split && own) {
          // the next such task has its parts in the same place: not before these are read
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.joined);
          ok = mbar_wait(&s.joined, joins++ & 1);
          ok = __all_sync(0xffffffffu, ok);
        }
      }
    }
  } else {
    fewer_regs<64>();
    if (warp < kMma) {
      // ---- queries and keys by two warps, values by two: of a tile this CTA's 64 keys, and its columns of the 128
      // values. (Each warp a quarter of both took 2000 cycles a tile, one instruction after the other.)
      const int half = warp & 1;
      constexpr int kK = 32, kV = 64, kVC = C::kVCols / 64;  // a warp's keys and values; their columns, by 64
      constexpr uint32_t kKShare = kK * D * 2, kVShare = kV * C::kVCols * 2;
      // lanes that copy, by four rows and 64 columns, or by boxes: where blocks are made of boxes of 8 rows or
      // more, a whole tile comes as boxes (a copy of four rows takes an SM 22 cycles, a box not much more)
      const uint32_t full0 = map_rank(&s.full[0], 0);
      const bool of_keys = warp < kLoad0 + 2;
      uint32_t slot = of_keys ? 0 : 1, parity = 1;  // the warp's next, and the parity of its emptying
      int filled = 0;                               // slots, of keys and values
      const auto wait = [&](uint64_t* b, uint32_t parity) { return ok = __all_sync(0xffffffffu, mbar_wait(b, parity)); };
      const auto next = [&] {
        slot += 2;
        if (slot >= SLOTS) slot -= SLOTS, parity ^= 1;
        filled += 2;
      };
      const auto row_of = [&](const KeyBlock& b, int req) {
        const int row = key_slot(p, b, req);
        return row < 0 ? rows_end : row;  // past the last row: zeros
      };
      if (of_keys) {
        const int b = maps.box_k, k4 = lane % 8, kc4 = lane / 8;  // by fours: which, and of which columns
        const int nb = b ? kK / b : 1, c_b = lane / nb, r_b = lane % nb * b;
        for (int n = 0; take(n); ++n) {
          const Seg& g = s.seg[n % kSegs];
          const int keys = g.keys, req = g.s, j0 = g.j0, j1 = g.j1, h = g.h, toks = g.toks, row0 = g.row0;
          const int key0 = rank * 64 + half * kK + lane;
          KeyBlock kb = key_block(p, req, j0 * KT + key0, keys);
#pragma unroll 1
          for (int j = j0; j < j1; ++j) {
            const int row = row_of(kb, req);
            if (j + 1 < j1) kb = key_block(p, req, (j + 1) * KT + key0, keys);
            if (!wait(&s.empty[slot], parity)) break;
            unsigned char* to = s.ring[slot] + half * kK * 128;
            const uint32_t bar = full0 + 8 * slot;
            if (lane == 0) arrive_expect_cluster(bar, kKShare);
            __syncwarp();
            if (b && (j + 1) * KT <= keys) {
              const int at = __shfl_sync(0xffffffffu, row, r_b);
              if (c_b < D / 64) tma_load_2d_pair(to + c_b * 8192 + r_b * 128, &maps.kb, h * D + c_b * 64, at, bar);
            } else {
              int at[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) at[e] = __shfl_sync(0xffffffffu, row, k4 * 4 + e);
              if (kc4 < D / 64) gather4_pair(to + kc4 * 8192 + k4 * 512, &maps.k, h * D + kc4 * 64, at, bar);
            }
            next();
            if (j == j0 && half == 0) {
              // the task's queries, beside its first keys: whole tokens, whatever comes after the last
              if (!wait(&s.q_empty, (n & 1) ^ 1)) break;
              if (lane == 0) {
                const uint32_t qbar = map_rank(&s.q_full, 0);
                int tiles = 0;
#pragma unroll
                for (int t = 0; t < TILES; ++t) tiles += (2 * t + rank) * tile_toks < toks;
                arrive_expect_cluster(qbar, tiles * D * 2 * tile_toks * G);
#pragma unroll
                for (int t = 0; t < TILES; ++t)
                  if ((2 * t + rank) * tile_toks < toks)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                      tma_load_3d_pair(s.q[t] + c * 16384, &maps.q, c * 64, h * G, row0 + (2 * t + rank) * tile_toks, qbar);
              }
              __syncwarp();
            }
          }
          if (!ok) break;
          if (lane == 0) mbar_arrive(&s.seg_empty[n % kSegs]);
        }
      } else {
        const int b = maps.box_v, v4 = lane % 16, vc4 = lane / 16;
        const int nb = b ? kV / b : 1, c_b = lane / nb, r_b = lane % nb * b;
        uint32_t edges = 0;  // edge tiles so far
        for (int n = 0; take(n); ++n) {
          const Seg& g = s.seg[n % kSegs];
          const int keys = g.keys, first_last = g.pos, req = g.s, j0 = g.j0, j1 = g.j1, toks = g.toks;
          const unsigned tag = g.tag;
          const int x0 = g.h * D + (D == 64 ? 32 : C::kVCols) * rank, key0 = half * kV + lane;
          KeyBlock lo = key_block(p, req, j0 * KT + key0, keys), hi = key_block(p, req, j0 * KT + key0 + 32, keys);
#pragma unroll 1
          for (int j = j0; j < j1; ++j) {
            const int row_lo = row_of(lo, req), row_hi = row_of(hi, req);
            if (j + 1 < j1) {
              lo = key_block(p, req, (j + 1) * KT + key0, keys);
              hi = key_block(p, req, (j + 1) * KT + key0 + 32, keys);
            }
            if (!wait(&s.empty[slot], parity)) break;
            unsigned char* to = s.ring[slot];
            const uint32_t bar = full0 + 8 * slot;
            const bool edge = j * KT + KT - 1 > first_last && toks > 1;  // some row does not see some of these keys
            const uint32_t to_bar = edge ? map_rank(&s.edge, rank) : bar;
            if (lane == 0) arrive_expect_cluster(to_bar, kVShare);
            __syncwarp();
            if (b && (j + 1) * KT <= keys) {
              const int a = __shfl_sync(0xffffffffu, row_lo, r_b & 31), c = __shfl_sync(0xffffffffu, row_hi, r_b & 31);
              if (c_b < kVC)
                tma_load_2d_pair(to + c_b * 16384 + (half * kV + r_b) * 128, &maps.vb, x0 + c_b * 64, r_b < 32 ? a : c, to_bar);
            } else {
              int at[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int from = v4 * 4 + e & 31;
                const int a = __shfl_sync(0xffffffffu, row_lo, from), c = __shfl_sync(0xffffffffu, row_hi, from);
                at[e] = v4 < 8 ? a : c;
              }
              if (vc4 < kVC) gather4_pair(to + vc4 * 16384 + half * kV * 128 + v4 * 512, &maps.v, x0 + vc4 * 64, at, to_bar);
            }
            if (edge) {
              // 0 x NaN: values that are not finite are taken out, and the rows that do see them told
              // by the column's first such key, in both CTAs
              if (!wait(&s.edge, edges++ & 1)) break;
              bool found = false;
              constexpr int kRow = C::kVCols / 8;  // 16-byte pieces
  #pragma unroll 8
              for (int e = lane; e < kV * kRow; e += 32) {
                const int row = half * kV + e / kRow, c = e % kRow;
                const uint4 v = *reinterpret_cast<const uint4*>(to + (c >> 3) * 16384 + row * 128 + (((c ^ row) & 7) << 4));
                // an exponent of ones, and one, is a carry into the sign's place
                const auto not_finite = [](uint32_t u) { return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                found |= (not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w)) != 0;
              }
              found = __any_sync(0xffffffffu, found);
              if (found) {
                constexpr int kOwn = D == 64 ? 32 : C::kVCols;
  #pragma unroll 1
                for (int e = lane; e < kV * C::kVCols; e += 32) {
                  const int row = half * kV + e / C::kVCols, c = e % C::kVCols;
                  uint16_t* q = reinterpret_cast<uint16_t*>(to + (c >> 6) * 16384 + row * 128 + ((((c >> 3) ^ row) & 7) << 4)) + (c & 7);
                  if ((*q & 0x7f80) == 0x7f80) {
                    if (c < kOwn) {
                      const unsigned word = tag << 12 | (unsigned)(4095 - (j * KT + row - first_last + 1024));
                      for (int a = 0; a < 2; ++a) atomic_max_cluster(map_rank(&s.poison[n % kSegs][kOwn * rank + c], a), word);
                    }
                    *q = 0;
                  }
                }
                if (lane < 2) atomic_max_cluster(map_rank(&s.flagged[n % kSegs], lane), tag);
                fence_proxy_async_smem();
              }
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(bar);
            }
            next();
          }
          if (!ok) break;
          if (lane == 0) mbar_arrive(&s.seg_empty[n % kSegs]);
        }
      }
      // No copy in flight when the CTA leaves: the first CTA waits for every slot that was filled. (Where a
      // wait has failed, for the last phases that were begun.)
      if (rank == 0)
        for (int e = max(0, filled - SLOTS); e < filled; ++e) mbar_wait(&s.full[e % SLOTS], e / SLOTS & 1);
    } else if (warp == kMma && rank == 0) {
      // ---- the products
      constexpr uint32_t is = idesc_bf16_f32(256, KT), io = idesc_bf16_f32(256, D) | kMnB;
      // the slots of the next keys and values, with their barriers' parities; those of the weights of each S
      uint32_t ks = 0, k_parity = 0, vs = 1, v_parity = 0, p_parity = 0, sn = 0;  // sn: S tiles, with one row tile
      const auto on_by_2 = [](uint32_t& slot, uint32_t& parity) {
        slot += 2;
        if (slot >= SLOTS) slot -= SLOTS, parity ^= 1;
      };
      // descriptors of the operands, as their low words change
      const uint64_t qd = sdesc_k_sw128(smem_u32(s.q[0])), kd = sdesc_k_sw128(smem_u32(s.ring[0])),
                     vd = sdesc_mn_sw128(smem_u32(s.ring[0]), 16384);
      // S of row tile t (into buffer b) from the keys in ring slot k
      const auto scores = [&](int t, int b, uint32_t k) {
        const uint64_t a = qd + t * (128 * D * 2 >> 4), kk = kd + k * (C::kSlotBytes >> 4);
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
          mma_bf16_pair(tmem + b * 128, a + ((e >> 2) * 16384 >> 4) + 2 * (e & 3), kk + ((e >> 2) * 8192 >> 4) + 2 * (e & 3), is, e > 0);
        mma_commit_pair(&s.s_full[b]);
      };
      const auto values = [&](int t, int b, uint32_t k, bool first, bool tell) {
        const uint64_t v = vd + k * (C::kSlotBytes >> 4);
#pragma unroll
        for (int e = 0; e < KT / 16; ++e)
          mma_bf16_ts_pair(tmem + C::kO + t * D, tmem + b * 128 + 8 * e, v + e * (2048 >> 4), io, !(first && e == 0));
        if (tell) mma_commit_pair(&s.o_done[TILES == 2 ? t : b]);
      };
      for (int n = 0; take(n); ++n) {
        const Seg& g = s.seg[n % kSegs];
        const int steps = g.j1 - g.j0, end0 = g.end[0] - g.j0, end1 = g.end[1] - g.j0;
        const bool split = TILES == 1 || g.split;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.seg_empty[n % kSegs]);
        ok = ok && mbar_wait(&s.q_full, n & 1);
        tc_fence_after();
        // The turns, PV of a tile and then an S, in the order that keeps the tensor cores busy while the
        // softmax works on another S: with two row tiles PV(0, e), S(0, e + 1), PV(1, e), S(1, e + 1), the
        // tile's softmax beside the other's products; where S alternates over the keys PV(e), S(e + 2).
        // One copy of their instructions: those that a task's end or beginning had for itself would
        // have to be fetched each time. One lane goes through a turn, waits and all: with the whole warp
        // waiting, the tensor cores had done their products each time before it came back with the next.
        const int turns = split ? steps + 2 : 2 * steps + 2;
#pragma unroll 1
        for (int x = 0; x < turns; ++x) {
          const int e = split ? x - 2 : (x >> 1) - 1, ahead = split ? e + 2 : e + 1;  // the tiles of PV and S
          const int t = TILES == 1 ? 0 : x & 1;                                       // row tile of O
          const int endt = split ? steps : t ? end1 : end0;
          const bool pv = e >= 0 && e < endt, sc = ahead < endt, begun = split || t == 0, last = split || t == 1;
          const int vb = TILES == 1 ? (sn + x) & 1 : t;  // the S of both: S(e + 2) comes where P(e) was
          if (e >= 0 && begun) ok = ok && mbar_wait(&s.full[vs], v_parity);
          if (pv) ok = ok && mbar_wait(&s.p_full[vb], p_parity >> vb & 1);
          tc_fence_after();
          __syncwarp();
          if (e >= 0) {
            if (elect_one()) {
              if (pv) values(t, vb, vs, e == 0 || (TILES == 2 && split && e == 1), TILES == 1 || !sc);
              if (last) mma_commit_pair(&s.empty[vs]);
            }
            __syncwarp();
          }
          if (ahead < steps) {
            if (begun) ok = ok && mbar_wait(&s.full[ks], k_parity);
            tc_fence_after();
            __syncwarp();
            if (elect_one()) {
              if (sc) scores(split ? 0 : t, vb, ks);
              if (last) mma_commit_pair(&s.empty[ks]);
              if (last && ahead == steps - 1) mma_commit_pair(&s.q_empty);
            }
            __syncwarp();
          }
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (pv) p_parity ^= 1u << vb;
          if (last) {
            if (e >= 0) on_by_2(vs, v_parity);
            if (ahead < steps) on_by_2(ks, k_parity);
          }
        }
        if (!ok) break;
        sn += steps;
      }
    } else if (warp == kSched && ok) {
      // ---- the pair's share, a part of a task at a time
      Walk<KT> w(p, plan, start);
      w.from(s.at, u0);
      long long u = u0;
      int j0 = w.j, n = 0;
      unsigned tag = 0;
      bool more = true;
      while (true) {
        // what the share begins with of a task, or ends with, may have no tiles
        while (more && j0 >= w.nt) {
          u = w.task + w.nt + p.tile_e;
          more = u < u1;
          if (more) w.next_task();
          j0 = 0;
        }
        ok = mbar_wait_cluster(&s.seg_empty[n % kSegs], (n / kSegs & 1) ^ 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          Seg& g = s.seg[n % kSegs];
          g.on = more;
          if (more) {
            const int t0 = w.i * p.tile_m, j1 = (int)min((long long)w.nt, j0 + (u1 - u));
            g.s = w.s;
            g.h = w.h;
            g.row0 = w.row0 + t0;
            g.toks = min(p.tile_m, w.n - t0);
            g.pos = w.ctx + t0;
            g.keys = w.ctx + w.n;
            g.j0 = j0;
            g.j1 = j1;
            for (int t = 0; t < 2; ++t) {
              const int first = 2 * t * tile_toks, last = min(g.toks, first + 2 * tile_toks) - 1;
              g.end[t] = t < TILES && first <= last ? max(j0, min(j1, (g.pos + last + KT) / KT)) : j0;
            }
            g.split = TILES == 2 && w.nt >= kSplit && g.toks <= 2 * tile_toks;
            if (g.split) g.end[0] = g.end[1] = j1;
            g.whole = w.task >= u0 && w.task + w.nt <= u1;
            g.slot = w.task >= u0;
            g.c0 = shares.owner(w.task);
            g.c1 = shares.owner(w.task + w.nt - 1);
            g.tag = ++tag;
          }
          mbar_arrive(&s.seg_full[n % kSegs]);
        }
        tag = __shfl_sync(0xffffffffu, tag, 0);
        ++n;
        if (!more) break;
        j0 = w.nt;  // on to the next task
      }
    }
  }
  if (on && !ok) {
    s.failed = 1;
    atomicCAS(p.error, 0u, (kStatusDeadline << 24) | (kAttnWait << 16) | (pair & 0xffff));
  }
  // every role of both CTAs is through: the softmax has waited for the last products, or a wait has failed
  tc_fence_before();
  __syncthreads();
  if (s.failed)  // the products in flight take microseconds
    for (int i = 0; i < 8; ++i) __nanosleep(1000000);
  cluster_sync();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc_pair(tmem, 512);
}

template <int D>
__global__ void __launch_bounds__(1024) plan_kernel(const AttnParams p) {
  __shared__ PlanScratch<1024> x;
  griddep_wait();
  griddep_launch_dependents();
  attn_plan<KT, 1024>(p, p.seq, p.start, x, true);
}

template <int D>
cudaError_t launch(AttnParams p, int grid, cudaStream_t s) {
  const size_t smem = sizeof(TileSmem<D>);
  cudaError_t e = opt_in<attn_tiles<D>>(smem);
  if (e != cudaSuccess) return e;
  TileMaps m = {};
  const int G = p.group.d;
  m.tokens = 128 / G;
  p.tile_m = Cfg<D>::kRows / 128 * m.tokens;
  // A task's own time (queries, first tile, join) in tiles of keys. More where all tasks have their keys split between
  // the row tiles, as a tile is one turn there and not two. With 3, 5, 8, 12 (us): 24 requests of 4 tokens over up to 6000, 40
  // heads of 128 on 8, 74, 71, 68, 69; 48 of 3 over up to 3000, 64 on 8, 99, 92, 88, 91; 4 of 32 over up to 2000, 64 on 8, 27, 26,
  // 25, 25; 12 of 8 over up to 12000, heads of 64, 38, 36, 37, 39; 96 of 4 over up to 1000 98, 97, 102, 105. Where they have not:
  // fresh prompts of 3000 tokens, heads of 64, 112, 116, 117, 127; 4 prompts of 1000, heads of 256, 77, 81, 83, 84; 24 of 8 over
  // up to 4000, heads of 256, 47, 47, 49, 49; with 1 these three 110, 84, 50.
  p.tile_e = Cfg<D>::kTiles == 2 && p.max_len <= 2 * m.tokens ? 8 : 3;
  p.tile_g = FastDiv::of(1);
  const long long rows = (long long)p.num_blocks * p.block.d, cols = (long long)p.Hkv * D;
  // the largest power of two of rows that blocks are made of, up to a load warp's
  for (int b = 8; b <= 64 && p.block.d % b == 0; b *= 2) {
    m.box_v = b;
    m.box_k = std::min(b, 32);
  }
  if (!attn_row_map(&m.k, p.k, rows, cols, p.ldk, 1) || !attn_row_map(&m.v, p.v, rows, cols, p.ldv, 1)) return cudaErrorInvalidValue;
  if (m.box_k && (!attn_row_map(&m.kb, p.k, rows, cols, p.ldk, m.box_k) || !attn_row_map(&m.vb, p.v, rows, cols, p.ldv, m.box_v)))
    return cudaErrorInvalidValue;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hkv * G, (cuuint64_t)p.tokens},
                   strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.ldq * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)m.tokens};
  if (!attn_encode(&m.q, p.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  if (p.seqs <= kAttnPlanned) p.seq = nullptr;
  if (p.seq) {
    const Launch one(dim3(1), 1024, 0, true, s);
    e = cudaLaunchKernelEx(&one.cfg, plan_kernel<D>, p);
    if (e != cudaSuccess) return e;
  }
  const Launch all(dim3(grid / 2 * 2), kNT, smem, true, s);
  return cudaLaunchKernelEx(&all.cfg, attn_tiles<D>, m, p);
}

}  // namespace

cudaError_t launch_attn_tiles(const AttnParams& p, int d, int grid, cudaStream_t s) {
  return d == 64 ? launch<64>(p, grid, s) : d == 128 ? launch<128>(p, grid, s) : launch<256>(p, grid, s);
}

}  // namespace gdn
