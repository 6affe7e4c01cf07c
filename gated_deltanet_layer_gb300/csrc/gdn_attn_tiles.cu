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
// Warps 0 - 7: the softmax, a row a thread, and the outputs. Warps 8 - 11: keys and values, 16 bytes
// a lane by cp.async, from any slot to where the swizzled operand has it, zeros past the
// last key. Warp 12: the products. With two row tiles the tensor cores work on one while
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
  uint64_t q_full, q_empty, full[C::kSlots], empty[C::kSlots], s_full[2], p_full[2], o_done[2], seg_done[2];
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
    *reinterpret_cast<uint4*>(o + c) = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
  }
}

// The CTA's share as a walk of segments: what is left of a task, or as much of it as is the
// CTA's.
template <int D>
struct Segments {
  using C = Cfg<D>;
  Walk<C::kM, C::kKT> w;
  long long u, u1;
  int j0, j1;  // key tiles of the segment
  __device__ __forceinline__ Segments(const AttnParams& p, const int4* seq, const long long* start, long long u0, long long u1,
                                      const int (&at)[4])
      : w(p, seq, start), u(u0), u1(u1) {
    w.from(at, u0);
    cut();
  }
  __device__ __forceinline__ void cut() {
    j0 = w.j;
    j1 = (int)min((long long)w.nt, j0 + (u1 - u));
  }
  __device__ __forceinline__ bool next() {
    u += j1 - j0;
    if (u >= u1) return false;
    w.next_task();
    cut();
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

template <int D>
__global__ void __launch_bounds__(kNT, 1) attn_tiles(const AttnParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  static_assert(sizeof(TileSmem<D>) <= 232448, "227 KB of shared memory a CTA");
  TileSmem<D>& s = *reinterpret_cast<TileSmem<D>*>(raw);
  constexpr int KT = C::kKT, SLOTS = C::kSlots;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&s.q_full, 4);
    mbar_init(&s.q_empty, 1);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&s.full[i], 4);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
      mbar_init(&s.o_done[i], 1);
      mbar_init(&s.seg_done[i], 4 * C::kTiles);
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
    attn_plan<C::kM, KT, kNT>(p, s.seq, s.start, s.scan, blockIdx.x == 0);
  }
  attn_zero_rows<kNT / 32>(p, seq, p.Hkv * p.group.d * D);
  const long long units = start[p.seqs];
  const Shares shares(units, (int)max(1LL, min((long long)gridDim.x, (units + 1) / 2)));
  const bool on = units > 0 && blockIdx.x < shares.ctas;
  const long long u0 = shares.first(blockIdx.x), u1 = shares.first(blockIdx.x + 1);
  if (warp == 0 && on) Walk<C::kM, KT>::find(p, seq, start, u0, s.at);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  bool ok = on;

  if (warp < kLoad0) {
    more_regs<200>();
    const int t = warp >> 2;  // row tile
    if (ok && t < C::kTiles) {
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const int r = (warp & 3) * 32 + lane;
      Segments<D> g(p, seq, start, u0, u1, s.at);
      int sn = 0, pv = 0;  // S tiles and PV products so far (of the row tile)
      int seg = 0;
      do {
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
            for (int c = 4; c < KT; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
            const float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
            if (__any_sync(0xffffffffu, tile_top > m + kSlack || m == -INFINITY)) {
              const float grown = fmaxf(m, tile_top), f = m == -INFINITY ? 0.f : ex2(m - grown);
              if (j > g.j0) {
                if (C::kTiles == 1) {  // S came before the last PV
                  ok = mbar_wait(&s.o_done[t], (pv - 1) & 1);
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
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < KT; c += 64) {
              uint32_t w[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float a = ex2(fmaf(x[c + 2 * i], p.scale_log2, -base)), e = ex2(fmaf(x[c + 2 * i + 1], p.scale_log2, -base));
                sum[i & 3] += a + e;
                w[i] = pack2(a, e);
              }
              tmem_st32(sc + c / 2, w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
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
          if (C::kTiles == 1 && end - g.j0 > 1) ok = mbar_wait(&s.o_done[t], (pv - 2) & 1);
          ok = ok && mbar_wait(&s.o_done[t], (pv - 1) & 1);
          tc_fence_after();
        }
        if (!(ok = named_all(1 + t, 128, ok))) break;
        const long long t0 = g.w.task, t1 = t0 + g.w.nt;
        const bool whole = t0 >= u0 && t1 <= u1;
        const long long slot = (2LL * blockIdx.x + (t0 >= u0)) * C::kM + t * 128;  // the part's first row
        const uint32_t tok = p.group.div(live ? R : 0), hd = (live ? R : 0) - tok * p.group.d;
        const long long row = g.w.row0 + tok, col = ((long long)g.w.h * p.group.d + hd) * D;
        const int* poison = s.poison[seg & 1];
        const bool flagged = s.dirty[seg & 1] != 0;
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
                float* part = p.part + (slot + r) * D + c;
#pragma unroll
                for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(part + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
              }
            }
          }
          if (!whole && live) p.part_ml[slot + r] = make_float2(m, l);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.seg_done[seg & 1]);
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
            // eight lanes a row
            for (int q = r >> 3; q < min(128, rows - first); q += 16) {
              float top = -INFINITY, sum = 0.f;
              for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(&p.part_ml[at(c) + q]).x);
              for (int c = c0; c <= c1; ++c) {
                const float2 ml = __ldcg(&p.part_ml[at(c) + q]);
                sum += ml.y * (ml.x == -INFINITY ? 0.f : ex2(ml.x - top));
              }
              const float in = sum == 0.f ? 0.f : 1.f / sum;
              const int RR = first + q;
              const uint32_t tk = p.group.div(RR), hh = RR - tk * p.group.d;
              for (int k = (r & 7) * 32; k < D; k += 256) {
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.f;
                for (int c = c0; c <= c1; ++c) {
                  const float pm = __ldcg(&p.part_ml[at(c) + q]).x, e = pm == -INFINITY ? 0.f : ex2(pm - top);
                  const float4* src = reinterpret_cast<const float4*>(p.part + (at(c) + q) * D + k);
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const float4 v = __ldcg(src + i);
                    o[4 * i] = fmaf(v.x, e, o[4 * i]);
                    o[4 * i + 1] = fmaf(v.y, e, o[4 * i + 1]);
                    o[4 * i + 2] = fmaf(v.z, e, o[4 * i + 2]);
                    o[4 * i + 3] = fmaf(v.w, e, o[4 * i + 3]);
                  }
                }
                put32(p, g.w.row0 + tk, ((long long)g.w.h * p.group.d + hh) * D + k, o, in);
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
      constexpr int kPieces = D / 8;                    // 16-byte pieces of a row
      constexpr int kPer = 32 / kPieces > 0 ? 32 / kPieces : 1;  // rows a warp copies at once
      constexpr int kKeys = KT / 4;                     // keys of a warp
      int n = 0;        // slots filled
      int arrived = 0;  // slots whose copies are done and told
      int qs = 0;       // tasks whose queries are loaded
      // Slot i is told once its copies have landed, two slots later.
      const auto tell = [&](int upto) {
        while (arrived < upto) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.full[arrived % SLOTS]);
          ++arrived;
        }
      };
      const auto flush = [&] {
        cp_async_wait_pending(0);
        tell(n);
      };
      // A wait before which everything that has been filled is told.
      const auto wait = [&](uint64_t* b, uint32_t parity) {
        if (!__all_sync(0xffffffffu, mbar_test(b, parity))) {
          flush();
          ok = __all_sync(0xffffffffu, mbar_wait(b, parity));
        }
        return ok;
      };
      if (ok) {
        Segments<D> g(p, seq, start, u0, u1, s.at);
        int seg = 0;
        const int c = lane % kPieces;
        const uint32_t piece0 = (c >> 3) * C::kChunk;
        do {
          if (seg >= 2) {
            // the flags are the task's before last until it is through with them
            wait(&s.seg_done[seg & 1], ((seg >> 1) - 1) & 1);
            if (!(ok = named_all(3, 128, ok))) break;
            const bool flagged = s.dirty[seg & 1] != 0;
            named_sync(3, 128);
            if (flagged) {
              for (int i = lt; i < D; i += 128) s.poison[seg & 1][i] = INT_MAX;
              if (lt == 0) s.dirty[seg & 1] = 0;
              named_sync(3, 128);
            }
          }
          const int keys = g.w.ctx + g.w.n, first_last = g.w.ctx + (int)p.group.div(g.w.i * C::kM);
          const long long col = (long long)g.w.h * D + c * 8;
          // of a warp's keys, a lane has the slot of one (heads of 256: of the first 16)
          KeyBlock kb = key_block(p, g.w.s, g.j0 * KT + wl * kKeys + lane % kKeys, keys);
          for (int j = g.j0; j < g.j1 && ok; ++j) {
            const int slot = key_slot(p, kb, g.w.s);
            if (j + 1 < g.j1) kb = key_block(p, g.w.s, (j + 1) * KT + wl * kKeys + lane % kKeys, keys);
#pragma unroll 1
            for (int which = 0; which < 2 && ok; ++which) {  // keys, values
              if (!wait(&s.empty[n % SLOTS], (n / SLOTS & 1) ^ 1)) break;
              const uint32_t dst = smem_u32(s.ring[n % SLOTS]) + piece0;
              const __nv_bfloat16* src = (which ? p.v : p.k) + col;
              const long long ld = which ? p.ldv : p.ldk;
#pragma unroll
              for (int r0 = 0; r0 < kKeys; r0 += kPer) {
                const int rr = r0 + lane / kPieces, row = wl * kKeys + rr;
                const int at = __shfl_sync(0xffffffffu, slot, rr);
                cp_async16_or_zero(dst + row * 128 + (((c ^ row) & 7) << 4), src + max(at, 0) * ld, at >= 0);
              }
              ++n;
              if (which && j * KT + KT - 1 > first_last && g.w.n > 1) {
                // some row does not see some of these keys: 0 x NaN. Values that are not finite are taken
                // out, and the rows that do see them told by the column's first such key.
                cp_async_commit();
                cp_async_wait_pending(0);
#pragma unroll 1
                for (int r0 = 0; r0 < kKeys; r0 += kPer) {
                  const int row = wl * kKeys + r0 + lane / kPieces;
                  unsigned char* at = s.ring[(n - 1) % SLOTS] + piece0 + row * 128 + (((c ^ row) & 7) << 4);
                  uint4 v = *reinterpret_cast<const uint4*>(at);
                  uint32_t u[4] = {v.x, v.y, v.z, v.w};
                  bool bad = false;
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    if ((u[i] & 0x7f80u) == 0x7f80u) {
                      atomicMin(&s.poison[seg & 1][c * 8 + 2 * i], j * KT + row);
                      u[i] &= 0xffff0000u;
                      bad = true;
                    }
                    if ((u[i] & 0x7f800000u) == 0x7f800000u) {
                      atomicMin(&s.poison[seg & 1][c * 8 + 2 * i + 1], j * KT + row);
                      u[i] &= 0xffffu;
                      bad = true;
                    }
                  }
                  if (bad) {
                    s.dirty[seg & 1] = 1;
                    *reinterpret_cast<uint4*>(at) = make_uint4(u[0], u[1], u[2], u[3]);
                  }
                }
                tell(n);
              } else {
                cp_async_commit();
                cp_async_wait_pending(2);
                tell(n - 2);
              }
              if (j == g.j0 && which == 0) {
                // the task's queries, beside its first keys; rows past the last are zero
                if (!wait(&s.q_empty, (qs & 1) ^ 1)) break;
                const int rows = g.w.n * (int)p.group.d;
#pragma unroll 1
                for (int x = lt; x < C::kM * kPieces; x += 128) {
                  const int row = x / kPieces, cc = x % kPieces, R = g.w.i * C::kM + row, rr = row & 127;
                  const bool live = R < rows;
                  const uint32_t tok = p.group.div(live ? R : 0), hd = (live ? R : 0) - tok * p.group.d;
                  cp_async16_or_zero(smem_u32(s.q[row >> 7]) + (cc >> 3) * (128 * 128) + rr * 128 + (((cc ^ rr) & 7) << 4),
                                     p.q + (g.w.row0 + tok) * p.ldq + ((long long)g.w.h * p.group.d + hd) * D + cc * 8, live);
                }
                cp_async_commit();
                flush();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.q_full);
                ++qs;
              }
            }
          }
          ++seg;
          ok = named_all(3, 128, ok);
        } while (ok && g.next());
      }
      flush();
    } else if (warp == kMma && ok) {
      // ---- the products
      Segments<D> g(p, seq, start, u0, u1, s.at);
      constexpr uint32_t is = idesc_bf16_f32(128, KT), io = idesc_bf16_f32(128, D) | kMnB;
      int n = 0, seg = 0, sn[2] = {0, 0}, pn[2] = {0, 0};
      const auto wait = [&](uint64_t* b, uint32_t parity) {
        ok = ok && mbar_wait(b, parity);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        return ok;
      };
      // S of row tile t (into buffer b) from the keys in ring slot k
      const auto scores = [&](int t, int b, int k) {
        if (elect_one()) {
          const uint32_t a = smem_u32(s.q[t]), kk = smem_u32(s.ring[k]);
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_bf16(tmem + b * C::kS, sdesc_k_sw128(a + (i >> 2) * (128 * 128)) + 2 * (i & 3),
                     sdesc_k_sw128(kk + (i >> 2) * C::kChunk) + 2 * (i & 3), is, i > 0);
          mma_commit(&s.s_full[b]);
        }
        __syncwarp();
      };
      const auto values = [&](int t, int b, int k, bool first) {
        if (elect_one()) {
          const uint32_t v = smem_u32(s.ring[k]);
#pragma unroll
          for (int i = 0; i < KT / 16; ++i)
            mma_bf16_ts(tmem + C::kO + t * D, tmem + b * C::kS + 8 * i, sdesc_mn_sw128(v + i * 2048, C::kChunk), io,
                        !(first && i == 0));
          mma_commit(&s.o_done[t]);
        }
        __syncwarp();
      };
      const auto release = [&](uint64_t* b) {
        if (elect_one()) mma_commit(b);
        __syncwarp();
      };
      const auto slot = [&](int i) { return i % SLOTS; };
      const auto filled = [&](int i) { return wait(&s.full[i % SLOTS], i / SLOTS & 1); };
      do {
        const int e[2] = {g.end(0), C::kTiles == 2 ? g.end(1) : g.j0};
        if (!wait(&s.q_full, seg & 1) || !filled(n)) break;
        const int steps = g.j1 - g.j0;
        if (C::kTiles == 2) {
          // ring slots of step i: keys n + 2 i, values n + 2 i + 1
          for (int t = 0; t < 2; ++t)
            if (e[t] > g.j0) scores(t, t, slot(n));
          release(&s.empty[slot(n)]);
          if (steps == 1) release(&s.q_empty);
          for (int i = 0; i < steps && ok; ++i) {
            const int j = g.j0 + i;
            for (int t = 0; t < 2 && ok; ++t) {
              if (j < e[t]) {
                if (!wait(&s.p_full[t], pn[t] & 1)) break;
                ++pn[t];
                if (!filled(n + 2 * i + 1)) break;
                values(t, t, slot(n + 2 * i + 1), i == 0);
              }
              if (j + 1 < e[t]) {
                if (!filled(n + 2 * i + 2)) break;
                scores(t, t, slot(n + 2 * i + 2));
              }
            }
            if (!ok || !filled(n + 2 * i + 1)) break;
            release(&s.empty[slot(n + 2 * i + 1)]);
            if (i + 1 < steps) {
              if (!filled(n + 2 * i + 2)) break;
              release(&s.empty[slot(n + 2 * i + 2)]);
              if (i + 2 == steps) release(&s.q_empty);
            }
          }
        } else {
          // S's buffers alternate over the whole share
          scores(0, sn[0]++ & 1, slot(n));
          release(&s.empty[slot(n)]);
          if (steps == 1) release(&s.q_empty);
          for (int i = 0; i < steps && ok; ++i) {
            if (i + 1 < steps) {
              if (!filled(n + 2 * i + 2)) break;
              scores(0, sn[0]++ & 1, slot(n + 2 * i + 2));
              release(&s.empty[slot(n + 2 * i + 2)]);
              if (i + 2 == steps) release(&s.q_empty);
            }
            const int b = pn[0] & 1;
            if (!wait(&s.p_full[b], (pn[0] >> 1) & 1)) break;
            ++pn[0];
            if (!filled(n + 2 * i + 1)) break;
            values(0, b, slot(n + 2 * i + 1), i == 0);
            release(&s.empty[slot(n + 2 * i + 1)]);
          }
        }
        n += 2 * steps;
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
  attn_plan<Cfg<D>::kM, Cfg<D>::kKT, 1024>(p, p.seq, p.start, x, true);
}

template <int D>
cudaError_t launch(AttnParams p, int grid, cudaStream_t s) {
  const size_t smem = sizeof(TileSmem<D>);
  cudaError_t e = opt_in<attn_tiles<D>>(smem);
  if (e != cudaSuccess) return e;
  if (p.seqs <= kAttnPlannedTiles) p.seq = nullptr;
  if (p.seq) {
    const Launch one(dim3(1), 1024, 0, true, s);
    e = cudaLaunchKernelEx(&one.cfg, plan_kernel<D>, p);
    if (e != cudaSuccess) return e;
  }
  const Launch all(dim3(grid), kNT, smem, true, s);
  return cudaLaunchKernelEx(&all.cfg, attn_tiles<D>, p);
}

}  // namespace

cudaError_t launch_attn_tiles(const AttnParams& p, int d, int grid, cudaStream_t s) {
  return d == 64 ? launch<64>(p, grid, s) : d == 128 ? launch<128>(p, grid, s) : launch<256>(p, grid, s);
}

}  // namespace gdn
