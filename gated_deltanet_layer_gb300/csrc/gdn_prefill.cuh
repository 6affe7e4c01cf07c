// Shared definitions of the prompt-side operators: launch parameters, the
// ragged batch's row and slot lookups, the error word.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

constexpr int kChunk = 64;  // tokens of one chunk of a sequence
// Longest sequence that the delta rule takes token by token. The two forms take the same
// time at 11 tokens (many requests of many heads) to 18 (few) (us, token by token / in
// chunks, for 64 requests of the full layer 302.5 / 388.2 at 8, 426.4 / 390.6 at 12, 550.0 /
// 391.3 at 16; for 8 requests of a shard 15.4 / 29.1, 21.4 / 29.0, 27.3 / 28.9 and 33.2 /
// 29.2 at 20).
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
};

__device__ __forceinline__ void record(unsigned int* error, uint32_t status, uint32_t what, uint32_t who) {
  atomicCAS(error, 0u, (status << 24) | (what << 16) | (who & 0xffff));
}

// Rows [b, e) of sequence s, always inside the batch; of the pad rows after
// the last sequence for s = seqs.
__device__ __forceinline__ void seq_rows(const Ragged& r, int s, int* b, int* e) {
  const int lo = __ldg(r.cu + s), hi = s < r.seqs ? __ldg(r.cu + s + 1) : r.tokens;
  *b = min(max(lo, 0), r.tokens);
  *e = min(max(hi, *b), r.tokens);
}

// The sequence's slots; false for padding (and for the pad rows, s = seqs).
// in <= 0: it starts from zero. `report`: one thread of the grid for each
// sequence records what is wrong with it.
__device__ __forceinline__ bool seq_slots(const Ragged& r, int s, bool report, int* in, int* out) {
  if (s >= r.seqs) return false;
  *in = __ldg(r.state_in + s);
  *out = __ldg(r.state_out + s);
  const int lo = __ldg(r.cu + s), hi = __ldg(r.cu + s + 1);
  const bool bad_rows = lo < 0 || hi < lo || hi > r.tokens || (s == 0 && lo != 0);
  if (report && bad_rows) record(r.error, kStatusIndex, kWhatOffsets, s);
  if (*out <= 0 || bad_rows) return false;
  const bool bad_slot = *in >= r.num_slots || *out >= r.num_slots, too_long = hi - lo > r.max_len;
  if (report && bad_slot) record(r.error, kStatusIndex, kWhatSlot, s);
  if (report && too_long) record(r.error, kStatusIndex, kWhatLength, s);
  return !bad_slot && !too_long;
}

// Chunks without a table: sequence s (and the pad rows, s = seqs) owns the
// chunk places from cu[s] / 64 + s on. The next one's are at least
// ceil(len / 64) further, because floor((x + n) / 64) - floor(x / 64) + 1 >=
// ceil(n / 64), so every chunk has a place of its own among tokens / 64 +
// seqs + 1, and a place is found from the offsets alone by bisection.
__host__ __device__ __forceinline__ int chunk_places(int tokens, int seqs) { return tokens / kChunk + seqs + 1; }
__device__ __forceinline__ int chunk_first_place(const Ragged& r, int s) {
  return min(max(__ldg(r.cu + s), 0), r.tokens) / kChunk + s;
}
// Place -> sequence (the last whose first place is at or before it). Every lane of a
// converged warp calls it: the lanes look at 32 sequences at a time, so the search is
// one step of dependent loads for up to 31 sequences and two for up to 1023.
__device__ __forceinline__ int chunk_seq(const Ragged& r, int place) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = r.seqs + 1;
  while (n > 1) {
    const int stride = (n + 31) / 32, at = lane * stride;
    const unsigned below = __ballot_sync(0xffffffffu, at < n && chunk_first_place(r, lo + min(at, n - 1)) <= place);
    const int last = below ? (31 - __clz(below)) * stride : 0;
    lo += last;
    n = min(stride, n - last);
  }
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

// Launchers, one for each operator's translation unit.
cudaError_t launch_conv(const ConvParams& p, cudaStream_t s);
// ws: delta_chunk_bytes() of device memory, 256-byte aligned.
cudaError_t launch_delta(const DeltaParams& p, int d, bool state_bf16, unsigned char* ws, cudaStream_t s);
cudaError_t launch_delta_chunks(const DeltaParams& p, int d, bool state_bf16, unsigned char* ws, cudaStream_t s);
size_t delta_chunk_bytes(long long tokens, long long seqs, int Hk, int Hv, int d);
cudaError_t launch_linear(const LinearParams& p, cudaStream_t s);
// Waits for the stream, reads the linear kernels' error word and clears it.
cudaError_t linear_error(unsigned int* word, cudaStream_t s);
cudaError_t launch_slot_map(const SlotParams& p, cudaStream_t s);

__device__ __forceinline__ float sigmoid_f(float t) { return 1.0f / (1.0f + expf(-t)); }
// log(1 + e^t), t itself above 20 (as in the decode step).
__device__ __forceinline__ float softplus_f(float t) { return t > 20.0f ? t : log1pf(expf(t)); }

}  // namespace gdn
