// Shared definitions of the prompt-side operators: launch parameters, the
// ragged batch's row and slot lookups, the error word.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

constexpr int kChunk = 64;  // tokens of one chunk of a sequence
// Longest sequence that the delta rule takes token by token. The two forms take the same
// time at 11 tokens (many requests of many heads) to 18 (few) (us, token by token / in
// chunks, for 64 requests of the full layer 304.1 / 383.2 at 8, 429.1 / 385.9 at 12, 553.1 /
// 387.8 at 16; for 8 requests of a shard 15.4 / 28.6, 21.3 / 28.7, 27.4 / 28.7 and 33.3 /
// 28.7 at 20).
constexpr int kRecurrentMax = 14;
// Up to this many sequences the chunked form starts the longest ones first, where they
// take more than one wave; with more of them the waves level out by themselves.
constexpr int kSorted = 128;

// What of an index error (bits 23..16 of the error word).
constexpr uint32_t kWhatSlot = 1, kWhatOffsets = 2, kWhatLength = 3, kWhatWait = 4;

struct Ragged {
  const int* cu;         // [seqs + 1]
  const int* state_in;   // [seqs]
  const int* state_out;  // [seqs]
  int seqs, tokens, num_slots, max_len;
  unsigned int* error;   // sticky word
  int* table;            // [seqs + 1] of the workspace: the rows' ends as they are taken, or nullptr (see seq_rows)
};

__device__ __forceinline__ void record(unsigned int* error, uint32_t status, uint32_t what, uint32_t who) {
  atomicCAS(error, 0u, (status << 24) | (what << 16) | (who & 0xffff));
}

// The offsets are the caller's, on the device: that they start at 0, do not decrease and end
// within the rows is known to nobody before the kernels run. So they are not taken as they
// are: sequence s has the rows [m_s, m_(s+1)), with m_0 = 0 and m_s the largest of cu[1..s]
// that lie within the rows, and the rows from m_seqs on are pad rows. These are in order
// whatever the offsets hold: every row has one owner, every sequence chunk places of its
// own, and a bad offset takes nothing from a sequence that is right. Offsets that are in
// order are their own m; a sequence whose offsets are not is padding.
// Up to kScanned sequences every warp works out the m it needs from all the offsets, four a
// lane; with more of them a kernel before leaves the m in a table. (The conv of single tokens
// of a small layer: 128 take 3.1 us scanned and 129 4.4 by the table; 400 take 5.2 by the
// table and, 32 offsets a lane, 7.1 scanned.)
constexpr int kScanned = 128;

// v, or 0 where it lies outside the rows.
__device__ __forceinline__ int offset_inside(const Ragged& r, int v) { return (unsigned)v > (unsigned)r.tokens ? 0 : v; }

// What the caller says of sequence s, or of the pad rows after the last one (s = seqs).
struct SeqIn {
  int lo, hi, in, out;
};
__device__ __forceinline__ SeqIn seq_in(const Ragged& r, int s) {
  if (s >= r.seqs) return SeqIn{__ldg(r.cu + s), r.tokens, 0, 0};
  return SeqIn{__ldg(r.cu + s), __ldg(r.cu + s + 1), __ldg(r.state_in + s), __ldg(r.state_out + s)};
}

// Rows [b, e) of sequence s. Every lane of a converged warp calls it.
__device__ __forceinline__ void seq_rows(const Ragged& r, int s, const SeqIn& q, int* b, int* e) {
  if (r.table) {
    *b = r.table[s];
    *e = s < r.seqs ? r.table[s + 1] : r.tokens;
  } else {
    int m = s > 0 ? offset_inside(r, q.lo) : 0;
#pragma unroll
    for (int k = 0; k < kScanned / 32; ++k) {
      const int i = 1 + (threadIdx.x & 31) + 32 * k;
      if (i < s) m = max(m, offset_inside(r, __ldg(r.cu + i)));
    }
    *b = __reduce_max_sync(0xffffffffu, m);
    *e = s < r.seqs ? max(*b, offset_inside(r, q.hi)) : r.tokens;
  }
}

// Whether sequence s with rows [b, e) is one to work on, not padding (nor the pad rows, s =
// seqs). in <= 0: it starts from zero. `report`: one thread of the grid for each sequence
// records what is wrong with it.
__device__ __forceinline__ bool seq_live(const Ragged& r, int s, const SeqIn& q, int b, int e, bool report) {
  if (s >= r.seqs) return false;
  if (report && (q.lo < 0 || q.hi < q.lo || q.hi > r.tokens || (s == 0 && q.lo != 0)))
    record(r.error, kStatusIndex, kWhatOffsets, s);
  if (q.out <= 0 || q.lo != b || q.hi != e) return false;
  const bool bad_slot = q.in >= r.num_slots || q.out >= r.num_slots, too_long = e - b > r.max_len;
  if (report && bad_slot) record(r.error, kStatusIndex, kWhatSlot, s);
  if (report && too_long) record(r.error, kStatusIndex, kWhatLength, s);
  return !bad_slot && !too_long;
}

// Chunk places: sequence s (and the pad rows, s = seqs), rows from b on, owns the
// chunk places from b / 64 + s on. The next one's are at least ceil(len / 64) further,
// because floor((x + n) / 64) - floor(x / 64) + 1 >= ceil(n / 64), so every chunk has a
// place of its own among tokens / 64 + seqs + 1, and its sequence is found from the offsets
// alone.
__host__ __device__ __forceinline__ int chunk_places(int tokens, int seqs) { return tokens / kChunk + seqs + 1; }
__device__ __forceinline__ int chunk_first_place(int s, int b) { return b / kChunk + s; }
// Place -> sequence (the last whose first place is at or before it; the first one's is 0)
// and its rows. Every lane of a converged warp calls it. WAITED: this grid has waited for the
// kernel that filled the table, so what L1 holds of it is new; else only L2 is sure to be (the
// grid before has waited, and then let this one start).
template <bool WAITED>
__device__ __forceinline__ int chunk_seq(const Ragged& r, int place, int* b, int* e) {
  const int lane = threadIdx.x & 31;
  const auto table = [&](int s) { return WAITED ? r.table[s] : __ldcg(r.table + s); };
  int lo = 0, n = r.seqs + 1;
  if (!r.table) {
    constexpr int kOf = kScanned / 32;  // a lane has m_s of s = kOf lane + 1 .. kOf lane + kOf
    static_assert(kOf == 4, "at() below");
    int m[kOf];
#pragma unroll
    for (int k = 0; k < kOf; ++k) {
      const int s = kOf * lane + k + 1;
      m[k] = s <= r.seqs ? offset_inside(r, __ldg(r.cu + s)) : 0;
    }
#pragma unroll
    for (int k = 1; k < kOf; ++k) m[k] = max(m[k], m[k - 1]);
    int top = m[kOf - 1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = max(top, __shfl_up_sync(0xffffffffu, top, o));  // a lane's own past the first
    int before = __shfl_up_sync(0xffffffffu, top, 1);
    if (lane == 0) before = 0;
#pragma unroll
    for (int k = 0; k < kOf; ++k) {
      const int s = kOf * lane + k + 1;
      m[k] = max(m[k], before);
      lo += __popc(__ballot_sync(0xffffffffu, s <= r.seqs && chunk_first_place(s, m[k]) <= place));
    }
    const auto at = [&](int s) {
      const int k = (s - 1) & 3;
      return __shfl_sync(0xffffffffu, k == 0 ? m[0] : k == 1 ? m[1] : k == 2 ? m[2] : m[3], (s - 1) >> 2);
    };
    const int begin = at(max(lo, 1)), end = at(min(lo + 1, max(r.seqs, 1)));
    *b = lo > 0 ? begin : 0;
    *e = lo < r.seqs ? end : r.tokens;
    return lo;
  }
  // 32 sequences at a time: two steps of dependent loads for up to 1023
  while (n > 1) {
    const int stride = (n + 31) / 32, i = lane * stride, s = lo + min(i, n - 1);
    const unsigned below = __ballot_sync(0xffffffffu, i < n && chunk_first_place(s, table(s)) <= place);
    const int last = below ? (31 - __clz(below)) * stride : 0;
    lo += last;
    n = min(stride, n - last);
  }
  *b = table(lo);
  *e = lo < r.seqs ? table(lo + 1) : r.tokens;
  return lo;
}

struct ConvParams {
  Ragged r;
  const __nv_bfloat16* x;
  long long ldx;
  const __nv_bfloat16* w;  // [C][4]
  __nv_bfloat16* state;    // [num_slots][C][3]
  __nv_bfloat16* out;
  long long ldo;
  int C;
};

struct DeltaParams {
  Ragged r;
  int Hk, Hv, group;
  const __nv_bfloat16* qkv;
  long long ldqkv;
  const __nv_bfloat16* z;  // nullptr: no gated norm
  long long ldz;
  const __nv_bfloat16* ba;
  long long ldba;
  const float* A_log;
  const __nv_bfloat16* dt_bias;
  const __nv_bfloat16* gnorm_w;
  void* state;
  __nv_bfloat16* out;
  long long ldo;
  float gnorm_eps, l2_eps, q_scale;
  int* order;  // [kSorted] of the workspace: the sequences by length, or nullptr: as they come
  int4* plan;  // [seqs] of the workspace: rows [x, y) of what the chunked form has to do, from slot z to slot w
};

struct LinearParams {
  int M, N, K;
  const __nv_bfloat16* x;
  long long ldx;
  const __nv_bfloat16* w;
  long long ldw;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  long long ldr;
  __nv_bfloat16* out;
  long long ldo;
  int act;
};

// linear_w4: as LinearParams, with the weights in 4 bits.
struct W4Params {
  int M, N, K, group;
  bool mx;  // E2M1 codes and e8m0 scales; else whole numbers, bf16 scales, zeros (nullptr: 8)
  const __nv_bfloat16* x;
  long long ldx;
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  long long ldr;
  __nv_bfloat16* out;
  long long ldo;
  int act, row_groups, shares;  // of a CTA: 16 weight rows each, and of the columns
};

struct SlotParams {
  int R, N, B, max_blocks, free_cap;
  const int* new_lens;
  const int* ctx_lens;
  int* table;
  const int* free_list;
  const int* free_count;
  int* free_count_out;
  int* cu;
  int* token_seq;
  int* token_pos;
  long long* slots;
  unsigned int* error;
};

// Launchers, one for each operator's translation unit. With a table launch_conv and
// launch_delta launch the kernel that fills it first.
cudaError_t launch_offsets(const Ragged& r, cudaStream_t s);
// A launch that may start while the kernel before it ends (programmatic stream
// serialisation), if `early`.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  Launch(dim3 grid, int threads, size_t smem, bool early, cudaStream_t s) {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = early;
  }
};
cudaError_t launch_conv(const ConvParams& p, cudaStream_t s);
// ws: delta_chunk_bytes() of device memory, 256-byte aligned.
cudaError_t launch_delta(const DeltaParams& p, int d, bool state_bf16, unsigned char* ws, cudaStream_t s);
cudaError_t launch_delta_chunks(const DeltaParams& p, int d, bool state_bf16, unsigned char* ws, cudaStream_t s);
size_t delta_chunk_bytes(long long tokens, long long seqs, int Hk, int Hv, int d);
cudaError_t launch_linear(const LinearParams& p, cudaStream_t s);
cudaError_t launch_linear_w4(const W4Params& p, cudaStream_t s);
// Waits for the stream, reads the linear kernels' error word and clears it.
cudaError_t linear_error(unsigned int* word, cudaStream_t s);
cudaError_t launch_slot_map(const SlotParams& p, cudaStream_t s);

__device__ __forceinline__ float sigmoid_f(float t) { return 1.0f / (1.0f + expf(-t)); }
// log(1 + e^t), t itself above 20 (as in the decode step).
__device__ __forceinline__ float softplus_f(float t) { return t > 20.0f ? t : log1pf(expf(t)); }

}  // namespace gdn
