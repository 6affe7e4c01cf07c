// Host side of the C ABI in include/gdn_prefill.h: config validation, argument
// checks and launches.
#include <new>

#include "gdn_prefill.cuh"
#include "gdn_prefill.h"

using namespace gdn;

struct gdn_prefill {
  gdn_prefill_config cfg;
  int device;
  unsigned char* ws;
};

namespace {

// The workspace: the error word, on lines of its own; the sequences' order; what the chunked
// form has to do; the tables of the conv's and the delta rule's offsets, where there can be
// more sequences than are scanned; then the chunks.
constexpr size_t kErrorBytes = 256;
constexpr size_t kOrderBytes = kSorted * 4;
size_t table_bytes(const gdn_prefill_config& c) {
  return c.max_seqs > kScanned ? ((size_t)(c.max_seqs + 1) * 4 + 255) / 256 * 256 : 0;
}
size_t plan_bytes(const gdn_prefill_config& c) { return ((size_t)c.max_seqs * 16 + 255) / 256 * 256; }
size_t head_bytes(const gdn_prefill_config& c) { return kErrorBytes + kOrderBytes + plan_bytes(c) + 2 * table_bytes(c); }

gdn_status validate(const gdn_prefill_config* c) {
  if (!c) return GDN_ERR_ARG;
  if (c->num_k_heads <= 0 || c->num_v_heads <= 0 || c->head_k_dim <= 0 || c->head_v_dim <= 0 || c->num_slots <= 0 ||
      c->max_tokens < 1 || c->max_seqs < 1)
    return GDN_ERR_ARG;
  if (c->ssm_dtype != GDN_STATE_F32 && c->ssm_dtype != GDN_STATE_BF16) return GDN_ERR_ARG;
  if (!(c->gated_norm_eps >= 0.f) || !(c->l2_eps >= 0.f) || !(c->q_scale == c->q_scale)) return GDN_ERR_ARG;
  if (c->conv_kernel != 4 || c->head_k_dim != c->head_v_dim) return GDN_ERR_UNSUPPORTED;
  if (c->head_k_dim != 64 && c->head_k_dim != 128) return GDN_ERR_UNSUPPORTED;
  if (c->num_v_heads % c->num_k_heads != 0 || c->num_v_heads > 1024) return GDN_ERR_UNSUPPORTED;
  if (c->max_tokens > (1 << 24) || c->max_seqs > 65535) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int channels(const gdn_prefill_config& c) { return 2 * c.num_k_heads * c.head_k_dim + c.num_v_heads * c.head_v_dim; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Memory that a call reads or writes: n bytes from p, or of a matrix the `width` bytes of rows
// `ld` bytes apart.
struct Span {
  const void* p;
  size_t n, ld = 0, width = 0;
};
Span matrix(const void* p, long long rows, long long ld, long long cols) {
  return Span{p, rows > 0 ? (size_t)((rows - 1) * ld + cols) * 2 : 0, (size_t)ld * 2, (size_t)cols * 2};
}
bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (x >= y + b.n || y >= x + a.n) return false;
  if (!a.ld || a.ld != b.ld) return true;
  // columns of the same rows: b's begin `at` bytes after a's in a row, or in the one before
  const size_t at = y >= x ? (y - x) % a.ld : (a.ld - (x - y) % a.ld) % a.ld;
  return at < a.width || at + b.width > a.ld;
}
template <int N>
bool overlaps_any(const Span& out, const Span (&in)[N]) {
  for (const Span& s : in)
    if (overlap(out, s)) return true;
  return false;
}

// GDN_ERR_ARG where the current device is not the handle's.
gdn_status check_device(const gdn_prefill* h) {
  int device;
  if (cudaGetDevice(&device) != cudaSuccess) return GDN_ERR_CUDA;
  return device == h->device ? GDN_OK : GDN_ERR_ARG;
}

gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// Checks common to the two calls over a ragged batch.
gdn_status check_ragged(const gdn_prefill* h, int32_t seqs, int32_t tokens, const int32_t* cu, const int32_t* in,
                        const int32_t* out) {
  if (!h || seqs < 0 || tokens < 0) return GDN_ERR_ARG;
  if (seqs > h->cfg.max_seqs || tokens > h->cfg.max_tokens) return GDN_ERR_ARG;
  if (!cu || !aligned(cu, 4)) return GDN_ERR_ARG;
  if (seqs > 0 && (!in || !out || !aligned(in, 4) || !aligned(out, 4))) return GDN_ERR_ARG;
  return check_device(h);
}

// which: the table, 0 the conv's, 1 the delta rule's
Ragged ragged(const gdn_prefill* h, int32_t seqs, int32_t tokens, int32_t max_len, const int32_t* cu, const int32_t* in,
              const int32_t* out, int which) {
  int* table = reinterpret_cast<int*>(h->ws + kErrorBytes + kOrderBytes + plan_bytes(h->cfg) + which * table_bytes(h->cfg));
  return Ragged{cu,   in, out, seqs, tokens, h->cfg.num_slots, max_len, reinterpret_cast<unsigned int*>(h->ws),
                seqs > kScanned ? table : nullptr};
}

// The table of the offsets (see seq_rows): a running maximum, 1024 sequences at a time.
__global__ void __launch_bounds__(1024) offsets_kernel(const Ragged r) {
  griddep_launch_dependents();
  __shared__ int tops[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
  for (int i0 = 0, k = 0; i0 <= r.seqs; i0 += 1024, k ^= 1) {
    const int i = i0 + threadIdx.x;
    int m = max(i > 0 && i <= r.seqs ? offset_inside(r, __ldg(r.cu + i)) : 0, before);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = max(m, __shfl_up_sync(0xffffffffu, m, o));
    if (lane == 31) tops[k][warp] = m;
    __syncthreads();  // two buffers: one barrier a turn is enough
    const int top = tops[k][lane];
    m = max(m, __reduce_max_sync(0xffffffffu, lane < warp ? top : 0));
    before = __reduce_max_sync(0xffffffffu, top);
    if (i <= r.seqs) r.table[i] = m;
  }
}

}  // namespace

cudaError_t gdn::launch_offsets(const Ragged& r, cudaStream_t s) {
  offsets_kernel<<<1, 1024, 0, s>>>(r);
  return cudaGetLastError();
}

extern "C" size_t gdn_prefill_workspace_bytes(const gdn_prefill_config* cfg) {
  if (validate(cfg) != GDN_OK) return 0;
  return head_bytes(*cfg) + delta_chunk_bytes(cfg->max_tokens, cfg->max_seqs, cfg->num_k_heads, cfg->num_v_heads, cfg->head_k_dim);
}

extern "C" gdn_status gdn_prefill_create(const gdn_prefill_config* cfg, void* workspace, size_t workspace_bytes,
                                         void* stream, gdn_prefill_t** out) {
  if (!out) return GDN_ERR_ARG;
  *out = nullptr;
  const gdn_status st = validate(cfg);
  if (st != GDN_OK) return st;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < gdn_prefill_workspace_bytes(cfg)) return GDN_ERR_ARG;
  int device;
  if (cudaGetDevice(&device) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemsetAsync(workspace, 0, kErrorBytes, (cudaStream_t)stream) != cudaSuccess) return GDN_ERR_CUDA;
  gdn_prefill* h = new (std::nothrow) gdn_prefill{*cfg, device, static_cast<unsigned char*>(workspace)};
  if (!h) return GDN_ERR_CUDA;
  *out = h;
  return GDN_OK;
}

extern "C" gdn_status gdn_prefill_conv(gdn_prefill_t* h, int32_t seqs, int32_t tokens, const void* x, int64_t ldx,
                                       const void* conv_w, const int32_t* cu_seqlens, const int32_t* state_in,
                                       const int32_t* state_out, void* conv_state, void* out, int64_t ldo, void* stream) {
  const gdn_status st = check_ragged(h, seqs, tokens, cu_seqlens, state_in, state_out);
  if (st != GDN_OK) return st;
  const int C = channels(h->cfg);
  if (!conv_w || !conv_state || (tokens > 0 && (!x || !out))) return GDN_ERR_ARG;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(conv_w, 16) || !aligned(conv_state, 16)) return GDN_ERR_ARG;
  if (ldx < C || ldo < C || ldx % 8 || ldo % 8) return GDN_ERR_ARG;
  const Span o = matrix(out, tokens, ldo, C), state{conv_state, (size_t)h->cfg.num_slots * C * 6};
  const Span in[] = {matrix(x, tokens, ldx, C), {conv_w, (size_t)C * 8}, {cu_seqlens, (size_t)(seqs + 1) * 4},
                     {state_in, (size_t)seqs * 4}, {state_out, (size_t)seqs * 4},
                     {h->ws, gdn_prefill_workspace_bytes(&h->cfg)}};
  if (overlaps_any(o, in) || overlap(o, state) || overlaps_any(state, in)) return GDN_ERR_ARG;
  if (seqs == 0 && tokens == 0) return GDN_OK;
  ConvParams p{};
  p.r = ragged(h, seqs, tokens, tokens, cu_seqlens, state_in, state_out, 0);
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.ldx = ldx;
  p.w = static_cast<const __nv_bfloat16*>(conv_w);
  p.state = static_cast<__nv_bfloat16*>(conv_state);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldo = ldo;
  p.C = C;
  return cuda_status(launch_conv(p, (cudaStream_t)stream));
}

extern "C" gdn_status gdn_prefill_delta(gdn_prefill_t* h, int32_t seqs, int32_t tokens, int32_t max_len, const void* qkv,
                                        int64_t ldqkv, const void* z, int64_t ldz, const void* ba, int64_t ldba,
                                        const float* A_log, const void* dt_bias, const void* gated_norm_w,
                                        const int32_t* cu_seqlens, const int32_t* state_in, const int32_t* state_out,
                                        void* ssm_state, void* core_out, int64_t ldcore, void* stream) {
  const gdn_status st = check_ragged(h, seqs, tokens, cu_seqlens, state_in, state_out);
  if (st != GDN_OK) return st;
  const gdn_prefill_config& c = h->cfg;
  const int C = channels(c), Hv = c.num_v_heads, cols = Hv * c.head_v_dim;
  if (max_len < 0 || !A_log || !dt_bias || !ssm_state || (z && !gated_norm_w)) return GDN_ERR_ARG;
  if (tokens > 0 && (!qkv || !ba || !core_out)) return GDN_ERR_ARG;
  if (!aligned(qkv, 16) || !aligned(z, 16) || !aligned(core_out, 16) || !aligned(ssm_state, 16)) return GDN_ERR_ARG;
  if (!aligned(ba, 2) || !aligned(A_log, 4) || !aligned(dt_bias, 2) || !aligned(gated_norm_w, 16)) return GDN_ERR_ARG;
  if (ldqkv < C || ldba < 2 * Hv || ldcore < cols || (z && ldz < cols)) return GDN_ERR_ARG;
  if (ldqkv % 8 || ldcore % 8 || (z && ldz % 8)) return GDN_ERR_ARG;
  const size_t sdt = c.ssm_dtype == GDN_STATE_BF16 ? 2 : 4;
  const Span o = matrix(core_out, tokens, ldcore, cols);
  const Span state{ssm_state, (size_t)c.num_slots * cols * c.head_k_dim * sdt};
  const Span in[] = {matrix(qkv, tokens, ldqkv, C), matrix(z, tokens, ldz, cols), matrix(ba, tokens, ldba, 2 * Hv),
                     {A_log, (size_t)Hv * 4}, {dt_bias, (size_t)Hv * 2},
                     {gated_norm_w, z ? (size_t)c.head_v_dim * 2 : 0}, {cu_seqlens, (size_t)(seqs + 1) * 4},
                     {state_in, (size_t)seqs * 4}, {state_out, (size_t)seqs * 4},
                     {h->ws, gdn_prefill_workspace_bytes(&c)}};
  if (overlaps_any(o, in) || overlap(o, state) || overlaps_any(state, in)) return GDN_ERR_ARG;
  if (seqs == 0 && tokens == 0) return GDN_OK;
  DeltaParams p{};
  p.r = ragged(h, seqs, tokens, max_len, cu_seqlens, state_in, state_out, 1);
  p.Hk = c.num_k_heads;
  p.Hv = Hv;
  p.group = Hv / c.num_k_heads;
  p.qkv = static_cast<const __nv_bfloat16*>(qkv);
  p.ldqkv = ldqkv;
  p.z = static_cast<const __nv_bfloat16*>(z);
  p.ldz = ldz;
  p.ba = static_cast<const __nv_bfloat16*>(ba);
  p.ldba = ldba;
  p.A_log = A_log;
  p.dt_bias = static_cast<const __nv_bfloat16*>(dt_bias);
  p.gnorm_w = static_cast<const __nv_bfloat16*>(gated_norm_w);
  p.state = ssm_state;
  p.out = static_cast<__nv_bfloat16*>(core_out);
  p.ldo = ldcore;
  p.gnorm_eps = c.gated_norm_eps;
  p.l2_eps = c.l2_eps;
  p.q_scale = c.q_scale;
  p.order = seqs <= kSorted && (long long)seqs * Hv > 152 ? reinterpret_cast<int*>(h->ws + kErrorBytes) : nullptr;
  p.plan = reinterpret_cast<int4*>(h->ws + kErrorBytes + kOrderBytes);
  return cuda_status(launch_delta(p, c.head_k_dim, c.ssm_dtype == GDN_STATE_BF16, h->ws + head_bytes(c),
                                  (cudaStream_t)stream));
}

extern "C" gdn_status gdn_prefill_check(gdn_prefill_t* h, void* stream, uint32_t* detail) {
  if (!h) return GDN_ERR_ARG;
  const gdn_status st = check_device(h);
  if (st != GDN_OK) return st;
  uint32_t word = 0;
  if (cudaMemcpyAsync(&word, h->ws, 4, cudaMemcpyDeviceToHost, (cudaStream_t)stream) != cudaSuccess ||
      cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (detail) *detail = word;
  if (!word) return GDN_OK;
  const uint32_t s = word >> 24;
  return s == GDN_ERR_DEADLINE || s == GDN_ERR_INDEX ? (gdn_status)s : GDN_ERR_FAILED;
}

extern "C" gdn_status gdn_prefill_reset(gdn_prefill_t* h, void* stream) {
  if (!h) return GDN_ERR_ARG;
  const gdn_status st = check_device(h);
  if (st != GDN_OK) return st;
  return cuda_status(cudaMemsetAsync(h->ws, 0, kErrorBytes, (cudaStream_t)stream));
}

extern "C" void gdn_prefill_destroy(gdn_prefill_t* h) { delete h; }

extern "C" gdn_status gdn_linear(int32_t rows, int32_t cols, int32_t inner, const void* x, int64_t ldx, const void* w,
                                 int64_t ldw, const void* bias, int32_t activation, const void* residual, int64_t ldr,
                                 void* out, int64_t ldo, void* stream) {
  if (rows < 0 || cols < 0 || inner < 1) return GDN_ERR_ARG;
  if (activation < GDN_ACT_NONE || activation > GDN_ACT_GELU_TANH) return GDN_ERR_ARG;
  if (rows == 0 || cols == 0) return GDN_OK;
  if (!x || !w || !out) return GDN_ERR_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 2) || !aligned(residual, 2) || !aligned(out, 2)) return GDN_ERR_ARG;
  if (ldx < inner || ldw < inner || ldo < cols || (residual && ldr < cols) || ldx % 8 || ldw % 8) return GDN_ERR_ARG;
  if (ldx >= (1LL << 38) || ldw >= (1LL << 38)) return GDN_ERR_UNSUPPORTED;  // a tile map's largest stride
  constexpr int32_t kEdge = INT32_MAX - 255;  // a tile may reach past the matrix, its coordinates are 32 bits
  if (rows > kEdge || cols > kEdge || inner > kEdge) return GDN_ERR_UNSUPPORTED;
  const Span o = matrix(out, rows, ldo, cols), r = matrix(residual, rows, ldr, cols);
  const Span in[] = {matrix(x, rows, ldx, inner), matrix(w, cols, ldw, inner), {bias, bias ? (size_t)cols * 2 : 0}};
  if (overlaps_any(o, in)) return GDN_ERR_ARG;
  if (overlap(o, r) && !(residual == out && ldr == ldo)) return GDN_ERR_ARG;
  LinearParams p{};
  p.M = rows;
  p.N = cols;
  p.K = inner;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.ldx = ldx;
  p.w = static_cast<const __nv_bfloat16*>(w);
  p.ldw = ldw;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.ldr = ldr;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldo = ldo;
  p.act = activation;
  return cuda_status(launch_linear(p, (cudaStream_t)stream));
}

extern "C" gdn_status gdn_linear_check(void* stream, uint32_t* detail) {
  uint32_t word = 0;
  if (linear_error(&word, (cudaStream_t)stream) != cudaSuccess) return GDN_ERR_CUDA;
  if (detail) *detail = word;
  return word ? GDN_ERR_DEADLINE : GDN_OK;
}

extern "C" gdn_status gdn_slot_map(int32_t requests, int32_t tokens, const int32_t* new_lens, const int32_t* context_lens,
                                   int32_t block_size, int32_t max_blocks, int32_t* block_table, const int32_t* free_list,
                                   int32_t free_cap, const int32_t* free_count, int32_t* free_count_out,
                                   int32_t* cu_seqlens, int32_t* token_seq, int32_t* token_pos, int64_t* slots,
                                   uint32_t* error, void* stream) {
  if (requests < 0 || tokens < 0 || block_size < 1 || max_blocks < 0 || free_cap < 0) return GDN_ERR_ARG;
  if (!free_count || !free_count_out || !cu_seqlens) return GDN_ERR_ARG;
  if (requests > 0 && (!new_lens || !context_lens)) return GDN_ERR_ARG;
  if (requests > 0 && max_blocks > 0 && !block_table) return GDN_ERR_ARG;
  if (free_cap > 0 && !free_list) return GDN_ERR_ARG;
  if (tokens > 0 && (!token_seq || !token_pos || !slots)) return GDN_ERR_ARG;
  const void* a4[] = {new_lens, context_lens, block_table, free_list, free_count, free_count_out, cu_seqlens,
                      token_seq, token_pos, error};
  for (const void* q : a4)
    if (!aligned(q, 4)) return GDN_ERR_ARG;
  if (!aligned(slots, 8)) return GDN_ERR_ARG;
  const size_t R = (size_t)requests, N = (size_t)tokens;
  const Span in[] = {{new_lens, R * 4}, {context_lens, R * 4}, {free_list, (size_t)free_cap * 4}, {free_count, 4}};
  const Span outs[] = {{block_table, R * max_blocks * 4}, {free_count_out, 4}, {cu_seqlens, (R + 1) * 4},
                       {token_seq, N * 4}, {token_pos, N * 4}, {slots, N * 8}, {error, error ? (size_t)4 : 0}};
  for (int i = 0; i < 7; ++i) {
    if (overlaps_any(outs[i], in)) return GDN_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return GDN_ERR_ARG;
  }
  SlotParams p{requests, tokens, block_size, max_blocks, free_cap, new_lens, context_lens, block_table, free_list,
               free_count, free_count_out, cu_seqlens, token_seq, token_pos, reinterpret_cast<long long*>(slots), error};
  return cuda_status(launch_slot_map(p, (cudaStream_t)stream));
}
