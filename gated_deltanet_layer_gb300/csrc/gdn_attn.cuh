// Shared definitions of the paged attention (gdn_attn_paged): launch parameters,
// the plan of its work, and the parts of rows that several CTAs work on.
//
// A task is (request, key/value head, tile of query rows). A tile is M of the request's n G rows, of
// which row r is token r / G, query head r % G of the head's G = Hq / Hkv; or, with G = 1, M tokens
// with all their heads. A task's
// units are the tiles of KT keys that its last row sees, and tile_e more for what a task
// takes beside its tiles (they come last, and nobody does anything in them). All tasks' units form one line, in
// the order request, head, row tile, key tile, and every CTA takes an equal, contiguous
// share of it, whatever the lengths: a CTA has whole tasks, and at its two ends
// parts of tasks that it shares with the CTAs beside it. The parts go to the workspace, and
// the CTA that finishes last joins them, in order.
#pragma once

#include "gdn_attn_shares.h"
#include "gdn_common.cuh"

namespace gdn {

// What of an index error (bits 23..16 of the error word).
constexpr uint32_t kAttnBlock = 1, kAttnOffsets = 2, kAttnLength = 3, kAttnWait = 4, kAttnContext = 5;

// Up to this many requests every CTA plans by itself, in shared memory; with more of
// them a kernel before leaves the plan in the workspace.
constexpr int kAttnPlanned = 128;

// n / d for 0 <= n < 2^31: division by an invariant integer as Granlund and Montgomery (1994) have it, by the
// high half of a product and a shift.
struct FastDiv {
  uint32_t d, mul, shift;
  __host__ static FastDiv of(uint32_t d) {
    uint32_t l = 0;
    while (l < 31 && (1u << l) < d) ++l;
    return FastDiv{d, (uint32_t)((((1ull << 32) * ((1ull << l) - d)) / d) + 1), l};
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

struct AttnParams {
  const int* cu;     // [seqs + 1]
  const int* ctx;    // [seqs]
  const int* table;  // [seqs][max_blocks]
  int seqs, tokens, max_len, max_blocks, num_blocks;
  int limit;         // most keys of a request
  FastDiv block;     // slots of a block
  FastDiv group;     // query heads of a key/value head
  int tile_m;        // M and G of the tasks' tiles
  int tile_e;        // units that a task takes beside its tiles
  FastDiv tile_g;
  int Hkv;
  const __nv_bfloat16* q;
  long long ldq;
  const __nv_bfloat16* k;
  long long ldk;
  const __nv_bfloat16* v;
  long long ldv;
  const __nv_bfloat16* gate;  // nullptr: none
  long long ldg;
  __nv_bfloat16* out;
  long long ldo;
  bool wide_out;              // rows of out are 32-byte aligned
  float scale_log2;           // scale times log2(e)
  float scale_pow2;           // the largest power of two that is not above it
  unsigned int* error;        // sticky word
  unsigned int* done;         // [2 grid] parts finished of the tasks whose first part is a CTA's; zero between calls
  float* part;                // [2 grid] sums of weights times values, M rows of D, relative to the part's maximum
  float2* part_ml;            // [2 grid][M] maximum (of scores times log2 e) and sum of weights
  int4* seq;                  // [seqs + 1] of the workspace: the plan, where a kernel before makes it
  long long* start;           // [seqs + 1]
};

__device__ __forceinline__ void attn_record(unsigned int* error, uint32_t what, uint32_t who) {
  atomicCAS(error, 0u, (kStatusIndex << 24) | (what << 16) | (who & 0xffff));
}

// An add that comes after all that the thread has written, and, behind a barrier, that its CTA has, and
// before all that it reads.
__device__ __forceinline__ unsigned atom_add_acq_rel_u32(unsigned* p, unsigned v) {
  unsigned old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// sum over i < n of floor((a i + b) / m) (a, b >= 0), by the steps of Euclid's algorithm: whole multiples of m are taken
// out, then the points below the line are counted along the other axis (Graham, Knuth and Patashnik, Concrete
// Mathematics, 3.5).
__device__ __forceinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
#pragma unroll 1
  while (n > 0) {
    if (a >= m) sum += (n - 1) * n / 2 * (a / m), a %= m;
    if (b >= m) sum += n * (b / m), b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return sum;
}

// Row tiles of a request and their key tiles. Tile i's last row is min((i + 1) M, n G) - 1, so
// all but the last tile see ctx + ceil((i + 1) M / G) keys, which are
// ceil((G ctx + (i + 1) M) / (G KT)) tiles.
template <int KT>
struct Tiles {
  __device__ __forceinline__ static int rows(const AttnParams& p, int n) { return (n * (int)p.tile_g.d + p.tile_m - 1) / p.tile_m; }
  __device__ __forceinline__ static int keys(const AttnParams& p, int n, int ctx, int i) {
    const uint32_t last = min((uint32_t)(i + 1) * p.tile_m, n * p.tile_g.d) - 1;
    return ((uint32_t)ctx + p.tile_g.div(last) + KT) / KT;
  }
  // units before row tile i (at most the last one)
  __device__ __forceinline__ static long long before(const AttnParams& p, int ctx, int i) {
    if (i == 0) return 0;
    const long long G = p.tile_g.d, m = G * KT;
    return floor_sum(i, m, p.tile_m, G * ctx + p.tile_m + m - 1) + (long long)i * p.tile_e;
  }
  __device__ __forceinline__ static long long total(const AttnParams& p, int n, int ctx) {
    const int t = rows(p, n);
    return before(p, ctx, t - 1) + keys(p, n, ctx, t - 1) + p.tile_e;
  }
};

template <int NT>
struct PlanScratch {
  int top[NT / 32];
  long long sum[NT / 32];
};

// The plan: seq[s] = {first row, new tokens (0: padding), context, -}, start[s] the units
// before request s, seq[seqs].x the first pad row and start[seqs] all units. The offsets are the
// caller's: row ends are the running maximum of the offsets that lie within the rows, and
// a request whose offsets are not its row ends is padding. A block of NT threads.
template <int KT, int NT>
__device__ __forceinline__ void attn_plan(const AttnParams& p, int4* seq, long long* start, PlanScratch<NT>& x, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int top = 0;
  long long units = 0;
#pragma unroll 1
  for (int base = 0; base < p.seqs; base += NT) {
    const int s = base + tid;
    const bool on = s < p.seqs;
    const int lo = on ? __ldg(p.cu + s) : 0, hi = on ? __ldg(p.cu + s + 1) : 0, c = on ? __ldg(p.ctx + s) : 0;
    int e = on && (unsigned)hi <= (unsigned)p.tokens ? hi : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) e = max(e, __shfl_up_sync(0xffffffffu, e, o));
    if (lane == 31) x.top[warp] = e;
    __syncthreads();
    int before = top;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      const int t = x.top[w];
      if (w < warp) before = max(before, t);
      top = max(top, t);
    }
    int b = __shfl_up_sync(0xffffffffu, e, 1);
    b = lane == 0 ? before : max(b, before);
    e = max(e, before);
    int n = on && lo == b && hi == e ? e - b : 0;
    const bool bad = on && (lo < 0 || hi < lo || hi > p.tokens || (s == 0 && lo != 0));
    const bool long_ = n > p.max_len, far = n > 0 && (c < 0 || (long long)c + n > p.limit);
    if (report) {
      if (bad) attn_record(p.error, kAttnOffsets, s);
      if (long_) attn_record(p.error, kAttnLength, s);
      if (far) attn_record(p.error, kAttnContext, s);
    }
    if (long_ || far) n = 0;
    const long long mine = n > 0 ? p.Hkv * Tiles<KT>::total(p, n, c) : 0;
    long long u = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, u, o);
      if (lane >= o) u += t;
    }
    if (lane == 31) x.sum[warp] = u;
    __syncthreads();
    long long first = units + u - mine;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      const long long t = x.sum[w];
      if (w < warp) first += t;
      units += t;
    }
    if (on) {
      seq[s] = make_int4(b, n, c, 0);
      start[s] = first;
    }
  }
  if (tid == 0) {
    seq[p.seqs] = make_int4(top, 0, 0, 0);
    start[p.seqs] = units;
  }
  __syncthreads();
}

// A walk over the units, task by task.
template <int KT>
struct Walk {
  const AttnParams& p;
  const int4* seq;
  const long long* start;
  long long task;  // the task's first unit
  int s, h, i, j;  // request, key/value head, row tile, key tile
  int nt, rows;    // key tiles of the task, row tiles of the request
  int row0, n, ctx;

  __device__ __forceinline__ Walk(const AttnParams& p, const int4* seq, const long long* start) : p(p), seq(seq), start(start) {}
  __device__ __forceinline__ void load() {
    const int4 q = seq[s];
    row0 = q.x;
    n = q.y;
    ctx = q.z;
    rows = Tiles<KT>::rows(p, n);
  }
  // Where unit u, one of start[seqs], is: at = {s, h, i, j}. A converged warp.
  __device__ __forceinline__ static void find(const AttnParams& p, const int4* seq, const long long* start, long long u, int (&at)[4]) {
    const int lane = threadIdx.x & 31;
    // the last of n candidates for which f holds (it does for the first, and for none after one for
    // which it does not), 32 at a time
    const auto last_of = [&](int n, auto f) {
      int lo = 0;
      while (n > 1) {
        const int stride = (n + 31) / 32, k = lane * stride;
        const unsigned held = __ballot_sync(0xffffffffu, k < n && (lane == 0 || f(lo + k)));
        const int last = (31 - __clz(held)) * stride;
        lo += last;
        n = min(stride, n - last);
      }
      return lo;
    };
    // the last request that starts at or before u: it has units
    const int s = last_of(p.seqs, [&](int k) { return start[k] <= u; });
    const int4 q = seq[s];
    const long long first = start[s], per = (start[s + 1] - first) / p.Hkv;
    const int h = (int)((u - first) / per);
    const long long in = u - first - h * per;
    const int i = last_of(Tiles<KT>::rows(p, q.y), [&](int k) { return Tiles<KT>::before(p, q.z, k) <= in; });
    if (lane == 0) at[0] = s, at[1] = h, at[2] = i, at[3] = (int)(in - Tiles<KT>::before(p, q.z, i));
  }
  __device__ __forceinline__ void from(const int (&at)[4], long long u) {
    s = at[0];
    load();
    h = at[1];
    i = at[2];
    j = at[3];
    nt = Tiles<KT>::keys(p, n, ctx, i);
    task = u - j;
  }
  __device__ __forceinline__ void next_task() {
    task += nt + p.tile_e;
    j = 0;
    if (++i == rows) {
      i = 0;
      if (++h == p.Hkv) {
        h = 0;
        do ++s;
        while (s < p.seqs && seq[s].y == 0);
        if (s >= p.seqs) return;
        load();
      }
    }
    nt = Tiles<KT>::keys(p, n, ctx, i);
  }
};

// Rows that no request works on: zero. Every warp of the grid calls it, of W a CTA: a warp
// looks at 32 requests at a time and writes every grid-th row of those that are padding.
template <int W>
__device__ __forceinline__ void attn_zero_rows(const AttnParams& p, const int4* seq, int cols) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int s0 = (threadIdx.x >> 5) * 32; s0 <= p.seqs; s0 += W * 32) {
    const int s = s0 + lane;
    int b = 0, e = 0;
    if (s <= p.seqs && (s == p.seqs || seq[s].y == 0)) {
      b = seq[s].x;
      e = s < p.seqs ? seq[s + 1].x : p.tokens;
    }
    unsigned todo = __ballot_sync(0xffffffffu, b < e);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int end = __shfl_sync(0xffffffffu, e, l);
      for (int r = __shfl_sync(0xffffffffu, b, l) + (int)((blockIdx.x + l) % gridDim.x); r < end; r += gridDim.x)
        for (int c = lane * 8; c < cols; c += 256) *reinterpret_cast<uint4*>(p.out + r * p.ldo + c) = make_uint4(0, 0, 0, 0);
    }
  }
}

// Key row of position pos (below the request's keys): its slot, or -1 where its block is
// outside the cache.
struct KeyBlock {
  int block, at;  // the table's entry, the slot in it; at < 0: no such key
};
__device__ __forceinline__ KeyBlock key_block(const AttnParams& p, int s, int pos, int keys) {
  if (pos >= keys) return KeyBlock{0, -1};
  const uint32_t b = p.block.div(pos);
  return KeyBlock{__ldg(p.table + (long long)s * p.max_blocks + b), (int)(pos - b * p.block.d)};
}
__device__ __forceinline__ int key_slot(const AttnParams& p, const KeyBlock& b, int s) {
  if (b.at < 0) return -1;
  if ((unsigned)b.block >= (unsigned)p.num_blocks) {
    attn_record(p.error, kAttnBlock, s);
    return -1;
  }
  return b.block * (int)p.block.d + b.at;
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

struct AppendParams {
  int tokens, Hq, Hkv, rotary, parts;  // parts: warps that share a token
  const __nv_bfloat16* q;
  long long ldq;
  const __nv_bfloat16* k;
  long long ldk;
  const __nv_bfloat16* v;
  long long ldv;
  const int* pos;
  const long long* slots;
  long long num_slots;
  const float* freq;
  const __nv_bfloat16* qw;
  const __nv_bfloat16* kw;
  float eps;
  __nv_bfloat16* q_out;
  long long ldqo;
  __nv_bfloat16* k_cache;
  long long ldkc;
  __nv_bfloat16* v_cache;
  long long ldvc;
  unsigned int* error;
};
cudaError_t launch_kv_append(AppendParams p, int d, bool pairs, cudaStream_t s);

// Tile maps: of the boxes of 64 columns of a matrix, and of a cache's rows.
bool attn_encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box);
bool attn_row_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld, int box_rows);

// Launchers. grid: CTAs of the launch (the workspace has two parts a CTA).
cudaError_t launch_attn_rows(const AttnParams& p, int d, int grid, cudaStream_t s);
cudaError_t launch_attn_tiles(const AttnParams& p, int d, int grid, cudaStream_t s);

}  // namespace gdn
